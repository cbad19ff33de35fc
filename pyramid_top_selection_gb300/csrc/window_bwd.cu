// Sliding-window attention with sinks, backward, on the fifth-generation tensor cores.
//
// P = exp(s q.k - lse), D = dO . O, dS = P (dO . v - D):  dQ = s dS K,  dK = s dS^T Q,  dV = P^T dO.
// Two kernels, each with its sums in tensor memory and no atomics, so the order of every sum is
// fixed: one walks the keys of a row tile (dQ: S, dP and dQ products), one the rows of a key tile
// (dK, dV: S^T, dP^T, dV and dK products). S and dP are formed twice, 7 products instead of 5; one
// kernel for all three would have to add dQ tiles into an fp32 buffer in memory, whose reductions
// bound the selected blocks' backward kernel (attn_bwd_tc.cu), in an order that changes.
//
// Rows are packed as in the forward (window_tc.cuh): a 128-row tile is (token, head) rows, P heads
// of the group together. dQ's kernel also writes -lse log2 e and D per row, in tile order, for the
// second kernel.
//
// The second kernel, and the one that adds partial sums, start while the one before them ends (programmatic
// launches): at 2 x 1999 rows of 8 heads the whole pass takes 46 us in a graph instead of 53.
//
// P and dS are rounded to bf16 for their products (2^-8 relative at most), sums are fp32. Every wait
// is bounded; one that gives up poisons what its CTA leaves unfinished.
#include <algorithm>

#include "device.cuh"
#include "internal.h"
#include "profile.h"
#include "tmap.h"
#include "window_tc.cuh"

namespace pisa {

size_t align256(size_t x);

namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 384;                  // warps 0-7 softmax and output, 8 (and 10) MMA, 9 loader, 11 items (dQ)
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kDrainNs = 1000000000ull;   // bound of the drain waits (work already issued)
constexpr uint64_t kPatient = 1ull << 40;      // the item warp outwaits the others, whose giving up it sees
constexpr uint32_t kNaN2 = 0x7fc07fc0u;        // two bf16 NaNs
constexpr int kDqCtas = 1024;                  // dQ's CTAs at most

struct BwdArgs {
  WinDims s;
  const int32_t* len;
  const float* lse;
  float *nlse, *delta;     // [B][Hkv][sets][Nqp][P]: -lse log2 e and D
  bf16 *dQ, *dK, *dV;
  float* part;             // fp32 partial sums of dV, dK: [slot][2][128][D]
  int32_t* status;
  int32_t* gave_up;        // dQ's CTAs: whether one of its waits gave up
  uint64_t wait_ns;
  int stall;
  int P, lp, tok, sets, Nqp;   // heads (2^lp) and tokens of a row tile, head sets of a group, padded Nq
  int n_tiles, n_heads, n_items;           // dQ: token tiles, (b, kv, set), items
  // dK, dV: key tiles, (b, kv), key tiles with sinks; token tiles of a chunk and chunks of a key tile, of
  // those without sinks (ct, nck) and with them (cts, ncs); items of the tiles with sinks, which come first
  int n_kt, n_bh, n_st, ct, nck, cts, ncs, n_snk;
};

// ------------------------------------------------------------------------------------------ dQ
template <int D>
struct DqSmem {
  static constexpr int KB = D / 64;
  static constexpr int TILE = KB * 128 * 128;
  static constexpr int NK = 3, NV = 2;               // a key tile is held from S to dQ, its values only for dP
  static constexpr int oQ = 0, oO = TILE, oK = 2 * TILE, oV = oK + NK * TILE;
  static constexpr int bytes = oV + NV * TILE;
};

// Work item w: a row tile. first[0]: its heads' place in the statistics' order.
__device__ __forceinline__ win::Item dq_item(const BwdArgs& a, int w) {
  const WinDims& s = a.s;
  const int tile = a.n_tiles - 1 - w / a.n_heads, hh = w % a.n_heads, set = hh % a.sets;
  win::Item it;
  it.b = hh / (s.Hkv * a.sets);
  it.kv = hh / a.sets % s.Hkv;
  it.h0 = it.kv * s.G + set * a.P;
  it.t0 = tile * a.tok;
  it.L = win::valid_len(a.len, it.b, s.N);
  const win::KeyList kl(s, it.L, s.off + it.t0, s.off + min(s.Nq, it.t0 + a.tok));
  it.lo = kl.lo;
  it.SP = kl.SP;
  it.n = (kl.n_cols + 127) >> 7;
  it.first[0] = (it.b * s.Hkv + it.kv) * a.sets + set;
  it.first[1] = it.last[0] = it.last[1] = 0;
  return it;
}

// TMEM: S (and dS in its place) of key tile n at 128 (n & 1), dP at 256, dQ at 384. One MMA warp
// issues dP(n) and the next tile's S, the other dQ += dS K as soon as dS is there, so that the
// tensor cores have a product at hand while the softmax warps turn S and dP into dS. (The barriers of
// dP, dS and dQ are two each, by the tile's parity: their waiters may be a tile apart.)
//
// D is dO . O from the forward's O: O's rows come by TMA as one more tile through the keys' ring, dO's
// are in shared memory for dP anyway, and the softmax threads form half a row's product each (a warp
// that formed D an item ahead from global memory bounded the kernel below windows of 1000 keys: 424 against
// 493 us at 512, 326 against 467 at 256, 4 x 16384 rows of 16 heads). But O's rounding to bf16 is felt by
// rows with few keys (windows under some 60: dQ and dK 1.5 to 2 times as far from the exact ones as
// their own rounding puts them, 1.42 times without it). An item of one or two key tiles, and so every
// short row, has all its dP in tensor memory at one time, the second tile's where dQ will be: there D
// is the fp32 sum of P dP itself.
//
// 4 x 16384 rows of 16 heads over 4 KV heads, d = 128: 690 us at a window of 1024 and 4 sinks (1.16
// PFLOP/s of its three products), 268 us for 8192 rows of 16 heads over 2, all causal (1.54); 640 and 256 us
// in short bursts.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dq_kernel(const BwdArgs a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap domap,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ CUtensorMap kmap32, const __grid_constant__ CUtensorMap vmap32,
                 const __grid_constant__ CUtensorMap omap) {
  using M = DqSmem<D>;
  extern __shared__ __align__(1024) unsigned char sm[];      // SW128 tiles first
  __shared__ __align__(8) uint64_t q_full, q_empty, k_full[M::NK], k_empty[M::NK], v_full[M::NV], v_empty[M::NV],
      s_full[2], dp_full[2], d_full, ds_full[2], dq_done[2], dq_last, dq_empty, drain[2], never;
  __shared__ win::ItemRing s_items;
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  __shared__ float s_sum[2][128];            // D of the rows, as two sums

  const WinDims& s = a.s;
  const int tid = threadIdx.x, warp = win::uniform(tid >> 5), lane = tid & 31;
  const uint32_t aQ = tc::su32(sm + M::oQ), aO = tc::su32(sm + M::oO), aK = tc::su32(sm + M::oK), aV = tc::su32(sm + M::oV);
  constexpr uint32_t kStage = M::TILE >> 4;                  // from one stage's descriptor to the next

  if (tid == 0) {
    tc::bar_init(&q_full, 1);
    tc::bar_init(&q_empty, 1);
    for (int k = 0; k < M::NK; ++k) {
      tc::bar_init(&k_full[k], 1);
      tc::bar_init(&k_empty[k], 1);
    }
    for (int k = 0; k < M::NV; ++k) {
      tc::bar_init(&v_full[k], 1);
      tc::bar_init(&v_empty[k], 1);
    }
    tc::bar_init(&s_full[0], 1);
    tc::bar_init(&s_full[1], 1);
    tc::bar_init(&dp_full[0], 1);
    tc::bar_init(&dp_full[1], 1);
    tc::bar_init(&d_full, 256);
    tc::bar_init(&ds_full[0], 256);
    tc::bar_init(&ds_full[1], 256);
    tc::bar_init(&dq_done[0], 1);
    tc::bar_init(&dq_done[1], 1);
    tc::bar_init(&dq_last, 1);
    tc::bar_init(&dq_empty, 256);
    tc::bar_init(&drain[0], 1);
    tc::bar_init(&drain[1], 1);
    win::ring_init(s_items, 11);
    tc::bar_init(&never, 1);
    tc::fence_bar_init();
    s_abort = 0;
    if (blockIdx.x == 0) *a.status = 0;      // nothing else writes it before the next kernel
  }
  if (warp == 0) tc::tmem_alloc(&tmem_base, 512);
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  if (tid == 0) win::launch_dependents();
  const uint32_t tm = tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return win::wait(bar, parity, &s_abort, a.wait_ns); };
  auto get = [&](int k) { return win::ring_get(s_items, k, &s_abort, a.wait_ns); };
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };

  if (warp == 9) {
    // ------------------------------------------------------------------ loader
    int n_k = 0, n_v = 0, n_q = 0;             // loads issued
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const win::Item it = get(i);
      if (it.n < 0) break;
      if (it.n == 0) continue;
      const win::KeyList kl(it.lo, it.SP);
      auto load = [&](int& k, uint64_t* full, uint64_t* empty, int ns, uint32_t base, int v0, const CUtensorMap* big,
                      const CUtensorMap* small) -> bool {
        const int st = k % ns;
        if (!wait(&empty[st], ((k / ns) & 1) ^ 1)) return false;
        ++k;
        if (lane == 0) {
          tc::bar_expect_tx(&full[st], M::TILE);
          const uint32_t dst = base + st * M::TILE;
          if (v0 >= kl.SP) {
#pragma unroll
            for (int kb = 0; kb < M::KB; ++kb)
              tc::tma_load4(dst + kb * (128 * 128), big, kb * 64, it.kv, kl.key(v0), it.b, &full[st]);
          } else {
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int kb = 0; kb < M::KB; ++kb)
                tc::tma_load4(dst + kb * (128 * 128) + r * (32 * 128), small, kb * 64, it.kv, kl.key(v0 + 32 * r), it.b, &full[st]);
          }
        }
        __syncwarp();
        return true;
      };
      if (!wait(&q_empty, (n_q & 1) ^ 1)) break;
      ++n_q;
      if (lane == 0) {
        tc::bar_expect_tx(&q_full, 2 * M::TILE);
#pragma unroll
        for (int kb = 0; kb < M::KB; ++kb) {
          tc::tma_load4(aQ + kb * (128 * 128), &qmap, kb * 64, it.h0, it.t0, it.b, &q_full);
          tc::tma_load4(aO + kb * (128 * 128), &domap, kb * 64, it.h0, it.t0, it.b, &q_full);
        }
      }
      __syncwarp();
      if (it.n > 2) {                          // O's rows take a key tile's place, before the first one
        const int st = n_k % M::NK;
        if (!wait(&k_empty[st], ((n_k / M::NK) & 1) ^ 1)) break;
        ++n_k;
        if (lane == 0) {
          tc::bar_expect_tx(&k_full[st], M::TILE);
#pragma unroll
          for (int kb = 0; kb < M::KB; ++kb)
            tc::tma_load4(aK + st * M::TILE + kb * (128 * 128), &omap, kb * 64, it.h0, it.t0, it.b, &k_full[st]);
        }
        __syncwarp();
      }
      for (int j = 0; ok && j < it.n; ++j)
        ok = load(n_k, k_full, k_empty, M::NK, aK, 128 * j, &kmap, &kmap32) &&
             load(n_v, v_full, v_empty, M::NV, aV, 128 * j, &vmap, &vmap32);
    }
    // whatever is still in flight lands before the CTA leaves
    for (int k = max(0, n_k - M::NK); k < n_k; ++k) tc::bar_wait(&k_full[k % M::NK], (k / M::NK) & 1, kDrainNs);
    for (int k = max(0, n_v - M::NV); k < n_v; ++k) tc::bar_wait(&v_full[k % M::NV], (k / M::NV) & 1, kDrainNs);
    if (n_q) tc::bar_wait(&q_full, (n_q - 1) & 1, kDrainNs);
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA, S and dP (the warp
    // together, one lane issuing: operands stay in uniform registers)
    const bool leader = win::elect();
    const uint32_t dQ = win::desc_lo(aQ), dO = win::desc_lo(aO), dK = win::desc_lo(aK), dV = win::desc_lo(aV);
    int n_q = 0, g = 0, kk = 0;                // items, key tiles, tiles through K's ring so far
    bool issued = false, ok = true;
    for (int i = 0; ok; ++i) {
      const int n = get(i).n;
      if (n < 0) break;
      if (n == 0) continue;
      if (a.stall && !wait(&never, 0)) { ok = false; break; }
      ok = wait(&q_full, n_q & 1);
      ++n_q;
      issued = true;
      kk += n > 2;
      auto issue_s = [&](int g) -> bool {      // where dS of two tiles ago has been read
        const int st = kk % M::NK;
        if (!wait(&k_full[st], (kk / M::NK) & 1)) return false;
        ++kk;
        if (g >= 2 && !wait(&dq_done[g & 1], ((g >> 1) - 1) & 1)) return false;
        tc::after_sync();
        if (leader) {
          win::product_ss<D>(tm + 128 * (g & 1), dQ, dK + st * kStage);
          tc::commit(&s_full[g & 1]);
        }
        __syncwarp();
        return true;
      };
      ok = ok && issue_s(g);
      for (int j = 0; ok && j < n; ++j, ++g) {
        const int st = g % M::NV;
        const bool aside = n == 2 && j == 1;   // dP(1) where dQ was, once the item before's has been read
        ok = wait(&v_full[st], (g / M::NV) & 1) &&
             (aside ? wait(&dq_empty, n_q & 1) : g == 0 || wait(&ds_full[(g - 1) & 1], ((g - 1) >> 1) & 1));   // dP has been read
        if (!ok) break;
        tc::after_sync();
        if (leader) {
          win::product_ss<D>(tm + (aside ? 384 : 256), dO, dV + st * kStage);
          tc::commit(&dp_full[g & 1]);
          tc::commit(&v_empty[st]);
          if (j + 1 == n) tc::commit(&q_empty);
        }
        __syncwarp();
        if (j + 1 < n) ok = issue_s(g + 1);
      }
    }
    if (issued) {
      if (leader) tc::commit(&drain[0]);
      __syncwarp();
      tc::bar_wait(&drain[0], 0, kDrainNs);
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------------ MMA, dQ
    const bool leader = win::elect();
    const uint32_t dK = win::desc_mn_lo(aK, 128 * 128);
    int n_q = 0, g = 0, kk = 0;
    bool issued = false, ok = true;
    for (int i = 0; ok; ++i) {
      const int n = get(i).n;
      if (n < 0) break;
      if (n == 0) continue;
      kk += n > 2;
      for (int j = 0; ok && j < n; ++j, ++g, ++kk) {
        const int st = kk % M::NK;
        ok = (j > 0 || wait(&dq_empty, (n_q & 1) ^ 1)) && wait(&ds_full[g & 1], (g >> 1) & 1) &&
             (j > 0 || n != 2 || wait(&ds_full[(g + 1) & 1], ((g + 1) >> 1) & 1));   // dP(1) has been read, too
        if (!ok) break;
        tc::after_sync();
        issued = true;
        if (leader) {
          win::product_ts<D, 64>(tm + 384, tm + 128 * (g & 1), dK + st * kStage, j > 0);
          tc::commit(&dq_done[g & 1]);
          tc::commit(&k_empty[st]);
          if (j + 1 == n) tc::commit(&dq_last);
        }
        __syncwarp();
      }
      ++n_q;
    }
    if (issued) {
      if (leader) tc::commit(&drain[1]);
      __syncwarp();
      tc::bar_wait(&drain[1], 0, kDrainNs);
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------------ items, decoded ahead of the other
    // roles; their rows' lse is asked into L2 meanwhile
    const int rounds = win::rounds_of(a.n_items);
    for (int k = 0; k <= rounds; ++k) {
      const int64_t w = k < rounds ? win::item_of(k, a.n_items) : -1;
      win::Item it{};
      if (w >= 0) it = dq_item(a, static_cast<int>(w));
      else it.n = -1;                                        // only the last round can miss a CTA
      bool ok = lane != 0 || win::ring_put(s_items, k, it, &s_abort, kPatient);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || w < 0) break;
      if (it.n == 0) continue;
      if (lane < 2 * a.P) {                                  // the first and the last token's lse of each head
        const int t = lane & 1 ? min(s.Nq, it.t0 + a.tok) - 1 : it.t0;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.lse + (static_cast<int64_t>(it.b) * s.Hq + it.h0 + (lane >> 1)) * s.Nq + t));
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax: row r, columns 64 g ..
    const int g = warp >> 2, r = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c1 = s.scale * kLog2e;
    int n_k = 0, n_q = 0, kk = 0, k_item = 0;
    auto lse_of = [&](const win::Item& x) -> float {
      const int rows = x.n > 0 ? min(128, (min(s.Nq, x.L - s.off) - x.t0) * a.P) : 0;
      return r < rows ? a.lse[(static_cast<int64_t>(x.b) * s.Hq + x.h0 + (r & (a.P - 1))) * s.Nq + x.t0 + (r >> a.lp)] : 0.f;
    };
    win::Item next = get(0);
    float lse_next = lse_of(next);
    for (;; ++k_item) {
      const win::Item it = next;
      const float nl = -kLog2e * lse_next;
      const int n = it.n, L = it.L;
      if (n < 0) break;
      const win::KeyList kl(it.lo, it.SP);
      const int i = it.t0 + (r >> a.lp), p = s.off + i, h = it.h0 + (r & (a.P - 1));
      const bool row = i < s.Nq && p < L;
      if (n == 0) {                                          // no row sees anything: dQ = 0
        if (g == 0 && i < s.Nq) {
          uint4* o = reinterpret_cast<uint4*>(a.dQ + ((static_cast<int64_t>(it.b) * s.Nq + i) * s.Hq + h) * D);
          for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0, 0, 0, 0);
        }
        next = get(k_item + 1);
        lse_next = lse_of(next);
        continue;
      }
      bool ok = true;
      // x = P, y = dP of key tile j; see: the visible columns, where some are not
      auto load = [&](int j, float (&x)[64], float (&y)[64], uint32_t (&see)[2], bool& masked) -> bool {
        const int k = n_k + j, v0 = 128 * j + 64 * g;
        bool ok = wait(&s_full[k & 1], (k >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc::after_sync();
        tc::tmem_ld64(tm + 128 * (k & 1) + 64 * g + lane_off, x);
        const int kb = kl.lo + v0 - kl.SP;
        const int hi = row ? p - kb : -1, lo = max(p - s.window + 1, kl.lo) - kb, sk = s.sinks - v0;
        see[0] = see[1] = 0xffffffffu;
        masked = !__all_sync(0xffffffffu, hi >= 63 && (lo <= 0 || sk >= 64));
        if (masked) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            see[q] = win::bit_range(0, hi - 32 * q) & (win::bit_range(lo - 32 * q, 31) | win::bit_range(0, sk - 1 - 32 * q));
        }
        const uint64_t cc = tc::pack2(c1, c1), ll = tc::pack2(nl, nl);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float y0, y1;
          tc::unpack2(tc::fma2(tc::pack2(x[c], x[c + 1]), cc, ll), y0, y1);
          x[c] = tc::ex2(y0);
          x[c + 1] = tc::ex2(y1);
        }
        ok = wait(&dp_full[k & 1], (k >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc::after_sync();
        tc::tmem_ld64(tm + (n == 2 && j == 1 ? 384 : 256) + 64 * g + lane_off, y);
        return true;
      };
      float x[64], y[64];
      uint32_t see[2];
      bool masked;
      // D: the sum of P dP, or dO . O of the tiles in shared memory
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      if (n <= 2) {
        for (int j = 0; ok && j < n; ++j) {
          ok = load(j, x, y, see, masked);
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!masked || (see[c >> 5] >> (c & 31)) & 1) sum[c & 3] = fmaf(x[c], y[c], sum[c & 3]);
        }
        if (!ok) break;
      } else {
        ok = wait(&q_full, n_q & 1) && wait(&k_full[kk % M::NK], (kk / M::NK) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        uint64_t acc[2] = {0, 0};
        const unsigned char* po = sm + M::oK + kk % M::NK * M::TILE + r * 128;
        const unsigned char* pd = sm + M::oO + r * 128;
        constexpr int HC = D / 16;                           // 16-byte pieces of half a row
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          const int pc = g * HC + c, at = (pc >> 3) * (128 * 128) + (((pc & 7) ^ (r & 7)) << 4);
          const uint4 o = *reinterpret_cast<const uint4*>(po + at), d = *reinterpret_cast<const uint4*>(pd + at);
          const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[e & 1] = tc::fma2(tc::pack2(__uint_as_float(ow[e] << 16), __uint_as_float(ow[e] & 0xffff0000u)),
                                  tc::pack2(__uint_as_float(dw[e] << 16), __uint_as_float(dw[e] & 0xffff0000u)), acc[e & 1]);
        }
        tc::unpack2(acc[0], sum[0], sum[1]);
        tc::unpack2(acc[1], sum[2], sum[3]);
      }
      s_sum[g][r] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc::bar_arrive(&d_full);
      ok = wait(&d_full, n_q & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      const float dl = s_sum[0][r] + s_sum[1][r];
      if (n > 2 && tid == 0) tc::bar_arrive(&k_empty[kk % M::NK]);
      kk += n > 2;
      if (g == 0 && row) {
        const int64_t at = (static_cast<int64_t>(it.first[0]) * a.Nqp + it.t0) * a.P + r;
        a.nlse[at] = nl;
        a.delta[at] = dl;
      }
      for (int j = 0; j < n; ++j) {
        ok = load(j, x, y, see, masked);
        if (!ok) break;
        const int k = n_k + j;
        const uint32_t tS = tm + 128 * (k & 1) + 64 * g + lane_off;
        const uint64_t dd = tc::pack2(-dl, -dl);
#pragma unroll
        for (int c = 0; c < 64; c += 2)
          tc::unpack2(win::mul2(tc::pack2(x[c], x[c + 1]), tc::add2(tc::pack2(y[c], y[c + 1]), dd)), x[c], x[c + 1]);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 64; ++c) x[c] = (see[c >> 5] >> (c & 31)) & 1 ? x[c] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t u[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) u[c] = pack_bf16(x[32 * q + 2 * c], x[32 * q + 2 * c + 1]);
          tc::tmem_st16(tS + 16 * q, u);
        }
        // keys at tokens >= len (the last tile's; S has read them) become zero: dS = 0 there, and dQ
        // must not meet what padding holds
        if (g == 0 && L < s.N && kl.key(128 * j + 127) >= L) {
          if (128 * j + r >= kl.SP && kl.key(128 * j + r) >= L)
            for (int c = 0; c < M::KB * 8; ++c)
              *reinterpret_cast<uint4*>(sm + M::oK + ((kk + j) % M::NK) * M::TILE + (c >> 3) * (128 * 128) + r * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          tc::fence_async_smem();
        }
        tc::tmem_wait_st();
        tc::before_sync();
        tc::bar_arrive(&ds_full[k & 1]);
      }
      if (!ok) break;
      n_k += n;
      kk += n;
      next = get(k_item + 1);
      lse_next = lse_of(next);
      // dQ of the item, scaled: row r's columns 64 g .. (shared memory is full, and Q's and dO's tiles
      // already take the next item's, so the rows go out from registers)
      ok = wait(&dq_last, n_q & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::after_sync();
      ++n_q;
      if (g < M::KB) {
        const int64_t row0 = ((static_cast<int64_t>(it.b) * s.Nq + it.t0) * s.Hq + it.h0) * D + 64 * g + 8 * (lane & 3);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float y[32];
          tc::tmem_ld32(tm + 384 + 64 * g + 32 * q + lane_off, y);
          uint32_t u[4][4];                                  // four 16-byte pieces of row r
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) u[c][k] = pack_bf16(s.scale * y[8 * c + 2 * k], s.scale * y[8 * c + 2 * k + 1]);
          win::transpose4(u, lane);                          // piece lane & 3 of four rows: 64 bytes of a row a store
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int rr = (r & ~3) + c;
            if (it.t0 + (rr >> a.lp) < s.Nq)
              *reinterpret_cast<uint4*>(a.dQ + row0 + (static_cast<int64_t>(rr >> a.lp) * s.Hq + (rr & (a.P - 1))) * D + 32 * q) =
                  make_uint4(u[c][0], u[c][1], u[c][2], u[c][3]);
          }
        }
      }
      tc::before_sync();
      tc::bar_arrive(&dq_empty);
    }
    if (aborted() && g == 0) {                               // the rows of the item at hand and of those left
      for (; k_item < win::rounds_of(a.n_items); ++k_item) {
        const int64_t w = win::item_of(k_item, a.n_items);
        if (w < 0) break;
        const win::Item it = dq_item(a, static_cast<int>(w));
        const int i = it.t0 + (r >> a.lp), h = it.h0 + (r & (a.P - 1));
        if (i >= s.Nq) continue;
        uint4* o = reinterpret_cast<uint4*>(a.dQ + ((static_cast<int64_t>(it.b) * s.Nq + i) * s.Hq + h) * D);
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(kNaN2, kNaN2, kNaN2, kNaN2);
      }
    }
  }
  tc::before_sync();
  __syncthreads();
  if (tid == 0) a.gave_up[blockIdx.x] = s_abort;
  if (s_abort) {                                             // the next kernel's gradients of these rows' keys are NaN
    for (int k = 0; k < win::rounds_of(a.n_items); ++k) {
      const int64_t w = win::item_of(k, a.n_items);
      if (w < 0) break;
      const win::Item it = dq_item(a, static_cast<int>(w));
      if (tid < 128 && it.t0 + (tid >> a.lp) < s.Nq)
        a.nlse[(static_cast<int64_t>(it.first[0]) * a.Nqp + it.t0) * a.P + tid] = __int_as_float(0x7fc00000);
    }
  }
  if (warp == 0) {
    tc::after_sync();
    tc::tmem_free(tm, 512);
  }
}

// --------------------------------------------------------------------------------------- dK, dV
template <int D>
struct DkvSmem {
  static constexpr int KB = D / 64;
  static constexpr int TILE = KB * 128 * 128;
  static constexpr int NQ = 3, NO = 2;               // Q is held from S^T to dK, dO from dP^T to dV
  static constexpr int oK = 0, oV = TILE, oQ = 2 * TILE, oO = oQ + NQ * TILE, oStat = oO + NO * TILE;
  static constexpr int oBar = oStat + 2 * 1024;      // per stage: 128 x -lse log2 e, 128 x D
  static constexpr int bytes = oBar + 256;           // d = 128: 231,680 of the 232,448 there are
};

struct DkvBars {
  uint64_t kv_full, q_full[3], q_empty[3], o_full[2], o_empty[2], st_full[2], st_empty[2], s_full, dp_full, p_full, ds_full,
      dv_done, dk_done, drain, never;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DkvBars) <= 256, "barrier block");

// The token tiles of key tile kt: the first token and how many tiles, for L valid tokens.
struct TokenRange {
  int i0, n;
  __host__ __device__ TokenRange(const WinDims& s, int tok, int L, int kt) {
    const int kb = 128 * kt;
    const int64_t see = static_cast<int64_t>(kb) + 127 + s.window;      // one past the last position of the band
    const int end = kb < s.sinks || see > L ? L : static_cast<int>(see);
    const int first = kb > s.off ? kb - s.off : 0;
    i0 = first & ~3;                                                    // 16-byte rows of the statistics
    const int last = kb < L ? end - s.off : 0;                          // a tile past the end has no key
    n = last > first ? (last - i0 + tok - 1) / tok : 0;
  }
};

struct DkvItem {
  int b, kv, kt, c, ct;            // chunk c, of ct token tiles, of the key tile's
  int64_t slot;                    // partial sums' slot, -1: the only chunk, written as it is
  __host__ __device__ DkvItem(const BwdArgs& a, int w) {
    const bool sink = w < a.n_snk;
    const int x = sink ? w : w - a.n_snk, tiles = sink ? a.n_st : a.n_kt - a.n_st;
    const int bh = x % a.n_bh;
    kt = x / a.n_bh % tiles + (sink ? 0 : a.n_st);
    c = x / a.n_bh / tiles;
    b = bh / a.s.Hkv;
    kv = bh % a.s.Hkv;
    ct = run_of(a, kt);
    slot = (sink ? a.ncs : a.nck) == 1 ? -1 : slot_of(a, kt, bh, c);
  }
  static __host__ __device__ int run_of(const BwdArgs& a, int kt) { return kt < a.n_st ? a.cts : a.ct; }
  // slots: sink tiles first ([kt][bh][ncs], where these are cut), then the others ([kt][bh][nck])
  static __host__ __device__ int64_t slot_of(const BwdArgs& a, int kt, int bh, int c) {
    if (kt < a.n_st) return (static_cast<int64_t>(kt) * a.n_bh + bh) * a.ncs + c;
    return (a.ncs > 1 ? a.n_snk : 0) + (static_cast<int64_t>(kt - a.n_st) * a.n_bh + bh) * a.nck + c;
  }
};

// One CTA per item: a tile of 128 keys of one KV head and a run of the row tiles that see it. TMEM:
// S^T (keys x rows; P^T in its place) at 0, dP^T (dS^T) at 128, dV at 256, dK at 256 + d. Per row
// tile n the MMA warp issues dV(n), S^T(n + 1), dK(n), dP^T(n + 1): the exponentials of one tile
// run under the dK and dP^T products, its dS under the next tile's dV and S^T. Each wait for a product
// that the next one overwrites the operand of is seen some 300 cycles after its issue; dK and dP^T a
// tile later would close these gaps, but hold two tiles' P in registers and spill (twice the time).
// 4 x 16384 rows of 16 heads over 4, a window of 1024, 4 sinks: 829 us, 1.29 PFLOP/s of its four products.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dkv_kernel(const BwdArgs a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap domap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap dkmap, const __grid_constant__ CUtensorMap dvmap, int dq_ctas) {
  using M = DkvSmem<D>;
  extern __shared__ __align__(1024) unsigned char sm[];      // the only shared memory: SW128 tiles first
  DkvBars& bar = *reinterpret_cast<DkvBars*>(sm + M::oBar);
  auto &kv_full = bar.kv_full, &s_full = bar.s_full, &dp_full = bar.dp_full, &p_full = bar.p_full, &ds_full = bar.ds_full,
       &dv_done = bar.dv_done, &dk_done = bar.dk_done, &drain = bar.drain,
       &never = bar.never;
  auto &q_full = bar.q_full, &q_empty = bar.q_empty;
  auto &o_full = bar.o_full, &o_empty = bar.o_empty, &st_full = bar.st_full, &st_empty = bar.st_empty;
  uint32_t& tmem_base = bar.tmem_base;
  int& s_abort = bar.abort;

  const WinDims& s = a.s;
  const int tid = threadIdx.x, warp = win::uniform(tid >> 5), lane = tid & 31;
  const uint32_t aK = tc::su32(sm + M::oK), aV = tc::su32(sm + M::oV), aQ = tc::su32(sm + M::oQ), aO = tc::su32(sm + M::oO);

  const DkvItem it(a, blockIdx.x);
  const int kb = 128 * it.kt, L = win::valid_len(a.len, it.b, s.N);
  const TokenRange tr(s, a.tok, L, it.kt);
  // this chunk's row tiles: token tile n / sets, head set n % sets
  const int tile0 = it.c * it.ct, n = win::uniform(max(0, min(it.ct, tr.n - tile0)) * a.sets);
  // This kernel starts while dQ's ends: what that wrote (statistics, status) is read after grid_wait only,
  // and one warp here waits for it in any case.
  if (warp == 11) {
    if (lane == 0) win::launch_dependents();
    if (blockIdx.x == 0) {
      win::grid_wait();
      int any = 0;
      for (int k = lane; k < dq_ctas; k += 32) any |= a.gave_up[k];
      if (__any_sync(0xffffffffu, any) && lane == 0) atomicOr(a.status, PISA_STATUS_TIMEOUT);
    }
  }
  if (n == 0 && it.slot >= 0) return;                        // the reduction knows which chunks are empty
  auto tile_tok = [&](int k) { return tr.i0 + (tile0 + k / a.sets) * a.tok; };
  auto tile_end = [&](int k) { return s.off + tile_tok(k) + a.tok; };    // one past its last position

  // the loads of row tile k (one lane; the stages it waits for are `wait`'s business)
  auto load_q = [&](int k) {
    const int sq = k % M::NQ;
    tc::bar_expect_tx(&q_full[sq], M::TILE);
#pragma unroll
    for (int x = 0; x < M::KB; ++x)
      tc::tma_load4(aQ + sq * M::TILE + x * (128 * 128), &qmap, x * 64, it.kv * s.G + k % a.sets * a.P, tile_tok(k), it.b, &q_full[sq]);
  };
  auto load_o = [&](int k) {
    const int so = k % M::NO;
    tc::bar_expect_tx(&o_full[so], M::TILE);
#pragma unroll
    for (int x = 0; x < M::KB; ++x)
      tc::tma_load4(aO + so * M::TILE + x * (128 * 128), &domap, x * 64, it.kv * s.G + k % a.sets * a.P, tile_tok(k), it.b, &o_full[so]);
  };
  auto load_stat = [&](int k) {
    const int ss = k & 1;
    const int64_t at = ((static_cast<int64_t>(it.b * s.Hkv + it.kv) * a.sets + k % a.sets) * a.Nqp + tile_tok(k)) * a.P;
    const uint32_t stat = tc::su32(sm + M::oStat) + ss * 1024;
    tc::bar_expect_tx(&st_full[ss], 1024);
    win::bulk_load(stat, a.nlse + at, 512, &st_full[ss]);
    win::bulk_load(stat + 512, a.delta + at, 512, &st_full[ss]);
  };
  if (warp == 9 && lane == 0) {        // the first loads run under the rest of the CTA's start
    tc::bar_init(&kv_full, 1);
    for (int k = 0; k < M::NQ; ++k) {
      tc::bar_init(&q_full[k], 1);
      tc::bar_init(&q_empty[k], 1);
    }
    for (int k = 0; k < M::NO; ++k) {
      tc::bar_init(&o_full[k], 1);
      tc::bar_init(&o_empty[k], 1);
      tc::bar_init(&st_full[k], 1);
      tc::bar_init(&st_empty[k], 8);
    }
    tc::bar_init(&s_full, 1);
    tc::bar_init(&dp_full, 1);
    tc::bar_init(&p_full, 256);
    tc::bar_init(&ds_full, 256);
    tc::bar_init(&dv_done, 1);
    tc::bar_init(&dk_done, 1);
    tc::bar_init(&drain, 1);
    tc::bar_init(&never, 1);
    tc::fence_bar_init();
    s_abort = 0;
    if (n > 0) {
      tc::bar_expect_tx(&kv_full, 2 * M::TILE);
#pragma unroll
      for (int x = 0; x < M::KB; ++x) tc::tma_load4(aK + x * (128 * 128), &kmap, x * 64, it.kv, kb, it.b, &kv_full);
      load_q(0);
#pragma unroll
      for (int x = 0; x < M::KB; ++x) tc::tma_load4(aV + x * (128 * 128), &vmap, x * 64, it.kv, kb, it.b, &kv_full);
      load_o(0);
      win::grid_wait();
      load_stat(0);
    }
  }
  if (warp == 0) tc::tmem_alloc(&tmem_base, 512);
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  const uint32_t tm = tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return win::wait(bar, parity, &s_abort, a.wait_ns); };
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };

  if (warp == 9) {
    // ------------------------------------------------------------------ loader
    if (lane == 0 && n > 0) {
      int n_q = 1, n_o = 1, n_st = 1;          // loads issued
      for (int k = 1; k < n && !aborted(); ++k) {
        if (!wait(&q_empty[k % M::NQ], ((k / M::NQ) & 1) ^ 1)) break;
        ++n_q;
        load_q(k);
        if (!wait(&o_empty[k % M::NO], ((k / M::NO) & 1) ^ 1)) break;
        ++n_o;
        load_o(k);
        if (!wait(&st_empty[k & 1], ((k >> 1) & 1) ^ 1)) break;
        ++n_st;
        load_stat(k);
      }
      // whatever is still in flight lands before the CTA leaves
      tc::bar_wait(&kv_full, 0, kDrainNs);
      for (int x = max(0, n_q - M::NQ); x < n_q; ++x) tc::bar_wait(&q_full[x % M::NQ], (x / M::NQ) & 1, kDrainNs);
      for (int x = max(0, n_o - M::NO); x < n_o; ++x) tc::bar_wait(&o_full[x % M::NO], (x / M::NO) & 1, kDrainNs);
      for (int x = max(0, n_st - 2); x < n_st; ++x) tc::bar_wait(&st_full[x & 1], (x >> 1) & 1, kDrainNs);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA (the warp together, one
    // lane issuing). What a product needs is waited for while the one before it still runs.
    if (n > 0) {
      const bool leader = win::elect();
      constexpr uint32_t kStage = M::TILE >> 4;              // from one stage's descriptor to the next
      const uint32_t dK = win::desc_lo(aK), dV = win::desc_lo(aV), dQ = win::desc_lo(aQ), dO = win::desc_lo(aO),
                     dQt = win::desc_mn_lo(aQ, 128 * 128), dOt = win::desc_mn_lo(aO, 128 * 128);   // as stored
      bool ok = wait(&kv_full, 0);
      if (ok && a.stall) ok = wait(&never, 0);
      const bool issued = ok;
      int sq = 0, pq = 0;                                    // Q's stage of the next row tile and its parity
      auto issue_s = [&](int k) -> bool {                    // S^T of row tile k
        if (!wait(&q_full[sq], pq)) return false;
        if (k > 0 && !wait(&dv_done, (k - 1) & 1)) return false;        // P^T has been read
        tc::after_sync();
        if (leader) {
          win::product_ss<D>(tm, dK, dQ + sq * kStage);
          tc::commit(&s_full);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](int k) -> bool {
        const int so = k % M::NO;
        if (!wait(&o_full[so], (k / M::NO) & 1)) return false;
        if (k > 0 && !wait(&dk_done, (k - 1) & 1)) return false;        // dS^T has been read
        tc::after_sync();
        if (leader) {
          win::product_ss<D>(tm + 128, dV, dO + so * kStage);
          tc::commit(&dp_full);
        }
        __syncwarp();
        return true;
      };
      ok = ok && issue_s(0) && issue_dp(0);
      for (int k = 0; ok && k < n; ++k) {
        const int so = k % M::NO, qk = sq;
        if (!wait(&p_full, k & 1)) break;
        tc::after_sync();
        if (leader) {
          win::product_ts<D, 64>(tm + 256, tm, dOt + so * kStage, k > 0);
          tc::commit(&dv_done);
          tc::commit(&o_empty[so]);
        }
        __syncwarp();
        if (++sq == M::NQ) {
          sq = 0;
          pq ^= 1;
        }
        if (k + 1 < n && !issue_s(k + 1)) break;
        if (!wait(&ds_full, k & 1)) break;
        tc::after_sync();
        if (leader) {
          win::product_ts<D, 64>(tm + 256 + D, tm + 128, dQt + qk * kStage, k > 0);
          tc::commit(&dk_done);
          tc::commit(&q_empty[qk]);
        }
        __syncwarp();
        if (k + 1 < n && !issue_dp(k + 1)) break;
      }
      if (issued) {
        if (leader) tc::commit(&drain);
        __syncwarp();
        tc::bar_wait(&drain, 0, kDrainNs);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax: key (lane) r, rows 64 g ..
    const int g = warp >> 2, r = tid & 127, key = kb + r;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c1 = s.scale * kLog2e;
    // positions that see this key: [key, see_end)
    const int64_t see_end = key >= L ? 0 : key < s.sinks ? L : min(static_cast<int64_t>(L), static_cast<int64_t>(key) + s.window);
    bool ok = true;
    for (int k = 0; k < n; ++k) {
      const int sq = k % M::NQ, ss = k & 1, pt0 = s.off + tile_tok(k);
      ok = wait(&st_full[ss], (k >> 1) & 1) && wait(&s_full, k & 1);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::after_sync();
      float x[64];
      const uint32_t tS = tm + 64 * g + lane_off;
      tc::tmem_ld64(tS, x);
      // column c is a row at position pt0 + c / P: visible iff lo <= c <= hi
      const int lo = max(-1, min(128, key - pt0)) * a.P - 64 * g;
      const int hi = static_cast<int>(max(int64_t(0), min(int64_t(128), see_end - pt0))) * a.P - 1 - 64 * g;
      uint32_t see[2] = {0xffffffffu, 0xffffffffu};
      const bool masked = !__all_sync(0xffffffffu, lo <= 0 && hi >= 63);
      if (masked) {
        see[0] = win::bit_range(lo, hi);
        see[1] = win::bit_range(lo - 32, hi - 32);
      }
      const float4* nl = reinterpret_cast<const float4*>(sm + M::oStat + ss * 1024 + 256 * g);
      const float4* dl = reinterpret_cast<const float4*>(sm + M::oStat + ss * 1024 + 512 + 256 * g);
      const uint64_t cc = tc::pack2(c1, c1);
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 l4 = nl[c / 4];
        float y0, y1;
        tc::unpack2(tc::fma2(tc::pack2(x[c], x[c + 1]), cc, tc::pack2(l4.x, l4.y)), y0, y1);
        x[c] = tc::ex2(y0);
        x[c + 1] = tc::ex2(y1);
        tc::unpack2(tc::fma2(tc::pack2(x[c + 2], x[c + 3]), cc, tc::pack2(l4.z, l4.w)), y0, y1);
        x[c + 2] = tc::ex2(y0);
        x[c + 3] = tc::ex2(y1);
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < 64; ++c) x[c] = (see[c >> 5] >> (c & 31)) & 1 ? x[c] : 0.f;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t u[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) u[c] = pack_bf16(x[32 * q + 2 * c], x[32 * q + 2 * c + 1]);
        tc::tmem_st16(tS + 16 * q, u);
      }
      // rows at positions >= len become zero in both tiles once S^T and dP^T have read them: P and dS
      // are 0 there, and dV and dK must not meet what padding holds
      if (L < s.N && tile_end(k) > L) {
        ok = wait(&dp_full, k & 1);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        const int base = g ? M::oO + k % M::NO * M::TILE : M::oQ + sq * M::TILE;
        if (pt0 + (r >> a.lp) >= L)
          for (int c = 0; c < M::KB * 8; ++c)
            *reinterpret_cast<uint4*>(sm + base + (c >> 3) * (128 * 128) + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        tc::fence_async_smem();
      }
      tc::tmem_wait_st();
      tc::before_sync();
      tc::bar_arrive(&p_full);
      ok = wait(&dp_full, k & 1);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::after_sync();
      const uint32_t tD = tm + 128 + 64 * g + lane_off;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float y[32];
        tc::tmem_ld32(tD + 32 * q, y);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 d4 = dl[8 * q + c / 4];
          float* p = x + 32 * q + c;
          tc::unpack2(win::mul2(tc::pack2(p[0], p[1]), win::sub2(tc::pack2(y[c], y[c + 1]), tc::pack2(d4.x, d4.y))), p[0], p[1]);
          tc::unpack2(win::mul2(tc::pack2(p[2], p[3]), win::sub2(tc::pack2(y[c + 2], y[c + 3]), tc::pack2(d4.z, d4.w))), p[2], p[3]);
        }
        if (masked) {                                        // what is not visible may be NaN in dP or D
#pragma unroll
          for (int c = 0; c < 32; ++c) x[32 * q + c] = (see[q] >> c) & 1 ? x[32 * q + c] : 0.f;
        }
        uint32_t u[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) u[c] = pack_bf16(x[32 * q + 2 * c], x[32 * q + 2 * c + 1]);
        tc::tmem_st16(tD + 16 * q, u);
      }
      tc::tmem_wait_st();
      tc::before_sync();
      tc::bar_arrive(&ds_full);
      if (lane == 0) tc::bar_arrive(&st_empty[ss]);
    }
    if (ok && n > 0) {
      ok = wait(&dk_done, (n - 1) & 1) && wait(&dv_done, (n - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      tc::after_sync();
    }
    ok = !__any_sync(0xffffffffu, !ok || aborted());
    // output: warps 0-3 dV, 4-7 dK (scaled), key r
    const float f = g ? s.scale : 1.f;
    const uint32_t tA = tm + 256 + D * g + lane_off;
    const float nan = __int_as_float(0x7fc00000);
    if (it.slot >= 0) {
      float* o = a.part + ((it.slot * 2 + g) * 128 + (r & ~3)) * D + 4 * (lane & 3);
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float x[32];
        if (ok) tc::tmem_ld32(tA + 32 * q, x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t u[4][4];                                  // four 16-byte pieces of row r, then one of four rows
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) u[c][k] = __float_as_uint(ok ? f * x[16 * h + 4 * c + k] : nan);
          win::transpose4(u, lane);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(o + c * D + 32 * q + 16 * h) = make_uint4(u[c][0], u[c][1], u[c][2], u[c][3]);
        }
      }
    } else if (!ok || n == 0) {
      const uint32_t v = ok ? 0u : kNaN2;
      if (key < s.N) {
        uint4* o = reinterpret_cast<uint4*>((g ? a.dK : a.dV) + ((static_cast<int64_t>(it.b) * s.N + key) * s.Hkv + it.kv) * D);
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(v, v, v, v);
      }
    } else {                                                 // through V's and K's shared memory
      const int base = g ? M::oK : M::oV;
#pragma unroll 1
      for (int x2 = 0; x2 < M::KB; ++x2) {
        float x[64];
        tc::tmem_ld64(tA + 64 * x2, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t u[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) u[k] = pack_bf16(f * x[8 * c + 2 * k], f * x[8 * c + 2 * k + 1]);
          *reinterpret_cast<uint4*>(sm + base + x2 * (128 * 128) + tc::sw128(r, 8 * c)) = make_uint4(u[0], u[1], u[2], u[3]);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          const int k0 = kb + 32 * (warp & 3);
          if (k0 < s.N)
            win::tma_store4(g ? &dkmap : &dvmap, 64 * x2, it.kv, k0, it.b,
                            tc::su32(sm + base) + x2 * (128 * 128) + (warp & 3) * (32 * 128));
          tc::bulk_commit();
        }
      }
      if (lane == 0) tc::bulk_wait<0>();
    }
  }
  tc::before_sync();
  __syncthreads();
  if (tid == 0 && s_abort) {
    win::grid_wait();
    atomicOr(a.status, PISA_STATUS_TIMEOUT);
  }
  if (warp == 0) {
    tc::after_sync();
    tc::tmem_free(tm, 512);
  }
}

// dK, dV of the key tiles that were cut into chunks: the chunks' partial sums in order.
// grid: (tiles x b kv, D / 4); a thread sums 4 elements.
template <int D>
__global__ void __launch_bounds__(256) window_dkv_sum_kernel(const BwdArgs a, int first_kt) {
  const WinDims& s = a.s;
  const int kt = first_kt + blockIdx.x / a.n_bh, bh = blockIdx.x % a.n_bh, b = bh / s.Hkv, kv = bh % s.Hkv;
  const int L = win::valid_len(a.len, b, s.N);
  const TokenRange tr(s, a.tok, L, kt);
  const int ct = DkvItem::run_of(a, kt), chunks = (tr.n + ct - 1) / ct;
  const int e = (blockIdx.y * 256 + threadIdx.x) * 4, which = e / (128 * D), r = e / D % 128, col = e % D;
  const int key = 128 * kt + r;
  if (key >= s.N) return;
  win::grid_wait();
  const float* p = a.part + (DkvItem::slot_of(a, kt, bh, 0) * 2 * 128) * D + e;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < chunks; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(c) * 2 * 128 * D);
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  bf16* o = (which ? a.dK : a.dV) + ((static_cast<int64_t>(b) * s.N + key) * s.Hkv + kv) * D + col;
  *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// The sizes that follow from a shape. Chunks: a key tile's rows are one item where the key tiles
// alone fill the GPU six times over; else (few heads, wide windows) runs of `ct` token tiles, whose
// partial sums a last kernel adds. Key tiles with sinks are seen by all rows behind them and have a run
// length of their own, `cts` (as long as the others', which a short window keeps short, they took 153 us of
// partial sums and 1054 us of dK/dV at 32768 tokens, 32 heads over 8, a window of 128 and 1024 sinks, now 24
// and 846). A tile that is cut has more rows than one run, so that there are less than
// twice as many runs as equal shares: under 2 x 17/16 x 912 of the tiles without sinks and as many of
// those with them, whatever the shape.
void plan(BwdArgs& a) {
  const WinDims& s = a.s;
  a.P = win::packed_heads(s.G);
  a.lp = win::log2_of(a.P);
  a.tok = 128 / a.P;
  a.sets = s.G / a.P;
  a.Nqp = (s.Nq + 3) & ~3;
  a.n_tiles = (s.Nq + a.tok - 1) / a.tok;
  a.n_heads = s.B * s.Hkv * a.sets;
  a.n_items = a.n_tiles * a.n_heads;
  a.n_kt = (s.N + 127) / 128;
  a.n_bh = s.B * s.Hkv;
  a.n_st = std::min(a.n_kt, (s.sinks + 127) / 128);
  const int64_t all = (s.Nq + 3 + a.tok - 1) / a.tok;                       // token tiles of every row
  const int64_t band = std::min(all, (int64_t(s.window) + 130 + a.tok - 1) / a.tok);
  const int64_t tiles = static_cast<int64_t>(a.n_kt) * a.n_bh, total = band * a.sets * tiles;
  constexpr int kSms = win::kPlanSms;
  // row tiles of an item: a sixth of a CTA's share, at least 16; a small problem (under 32 a CTA) whose
  // key tiles leave CTAs idle is cut into as many equal runs as there are CTAs for
  int64_t want = std::max<int64_t>(16, total / (kSms * 6));
  const bool small = total < kSms * 32 && tiles < kSms;
  if (small) want = (band * a.sets + kSms / tiles - 1) / (kSms / tiles);
  a.ct = static_cast<int>(std::min(band, (want + a.sets - 1) / a.sets));
  a.nck = static_cast<int>((band + a.ct - 1) / a.ct);
  a.cts = a.ct;
  a.ncs = a.nck;
  a.n_snk = 0;
  if (a.n_st > 0) {              // the same shares, of all the work; in a small problem half a CTA's, if not the others' run
    const int64_t sink_tiles = static_cast<int64_t>(a.n_st) * a.n_bh;
    const int64_t work = (band * (tiles - sink_tiles) + all * sink_tiles) * a.sets;
    const int64_t run = small ? std::max(want, work / (kSms * 2)) : std::max<int64_t>(16, work / (kSms * 6));
    a.cts = static_cast<int>(std::min(all, (run + a.sets - 1) / a.sets));
    a.ncs = static_cast<int>((all + a.cts - 1) / a.cts);
    a.n_snk = a.n_st * a.n_bh * a.ncs;
  }
}

int64_t part_slots(const BwdArgs& a) {
  const int64_t sink = a.ncs > 1 ? a.n_snk : 0;
  const int64_t rest = a.nck > 1 ? static_cast<int64_t>(a.n_kt - a.n_st) * a.n_bh * a.nck : 0;
  return sink + rest;
}

// A launch that starts while the kernel before it ends (which it waits for itself, with grid_wait).
struct Behind {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  Behind(dim3 grid, int threads, int smem, cudaStream_t st) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  Behind(const Behind&) = delete;
};

template <int D>
int bwd_launch(const BwdArgs& a, const CUtensorMap* m, cudaStream_t st) {
  static win::Ready dq_ready, dkv_ready;
  if (int e = dq_ready(window_dq_kernel<D>, DqSmem<D>::bytes)) return e;
  if (int e = dkv_ready(window_dkv_kernel<D>, DkvSmem<D>::bytes)) return e;
  const int dq_ctas = std::min({a.n_items, sm_count(), kDqCtas});
  {
    ProfScope ps(st, "window_dq");
    window_dq_kernel<D><<<dq_ctas, kThreads, DqSmem<D>::bytes, st>>>(a, m[0], m[1], m[2], m[3], m[4], m[5], m[8]);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  {
    ProfScope ps(st, "window_dkv");
    const int items = a.n_snk + (a.n_kt - a.n_st) * a.n_bh * a.nck;
    const Behind b(dim3(items), kThreads, DkvSmem<D>::bytes, st);
    e = cudaLaunchKernelEx(&b.cfg, window_dkv_kernel<D>, a, m[0], m[1], m[2], m[3], m[6], m[7], dq_ctas);
  }
  if (e != cudaSuccess) return e;
  const int first = a.ncs > 1 ? 0 : a.n_st, end = a.nck > 1 ? a.n_kt : a.n_st;
  if (first < end) {
    ProfScope ps(st, "window_dkv_sum");
    const Behind b(dim3((end - first) * a.n_bh, D / 4), 256, 0, st);
    e = cudaLaunchKernelEx(&b.cfg, window_dkv_sum_kernel<D>, a, first);
  }
  return e;
}

}  // namespace

WinBwdWs window_bwd_ws(const WinDims& s) {
  BwdArgs a{};
  a.s = s;
  plan(a);
  const size_t rows = align256(static_cast<size_t>(s.B) * s.Hq * a.Nqp * 4 + 512);   // a tile's read may pass the end
  WinBwdWs w{};
  w.status = 0;
  w.gave_up = 256;
  w.nlse = w.gave_up + kDqCtas * 4;
  w.delta = w.nlse + rows;
  w.part = w.delta + rows;
  w.total = w.part + static_cast<size_t>(part_slots(a)) * 2 * 128 * s.d * 4;
  return w;
}

int launch_window_bwd(const WinDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                      const void* dO, const int32_t* len, void* dQ, void* dK, void* dV, char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WinBwdWs w = window_bwd_ws(s);
  BwdArgs a{};
  a.s = s;
  plan(a);
  a.len = len;
  a.lse = lse;
  a.nlse = reinterpret_cast<float*>(ws + w.nlse);
  a.delta = reinterpret_cast<float*>(ws + w.delta);
  a.dQ = static_cast<bf16*>(dQ);
  a.dK = static_cast<bf16*>(dK);
  a.dV = static_cast<bf16*>(dV);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.status = reinterpret_cast<int32_t*>(ws);
  a.gave_up = reinterpret_cast<int32_t*>(ws + w.gave_up);
  a.wait_ns = wait_limit_ns();
  a.stall = test_stall();
  const int64_t hd = static_cast<int64_t>(s.Hq) * s.d, kd = static_cast<int64_t>(s.Hkv) * s.d;
  CUtensorMap m[9];
  if (int e = win::token_map(&m[0], Q, s.B, s.Nq, s.Hq, s.d, s.qs, a.P, a.tok)) return e;
  if (int e = win::token_map(&m[1], dO, s.B, s.Nq, s.Hq, s.d, hd, a.P, a.tok)) return e;
  if (int e = win::token_map(&m[2], K, s.B, s.N, s.Hkv, s.d, s.ks, 1, 128)) return e;
  if (int e = win::token_map(&m[3], V, s.B, s.N, s.Hkv, s.d, s.vs, 1, 128)) return e;
  if (int e = win::token_map(&m[4], K, s.B, s.N, s.Hkv, s.d, s.ks, 1, 32)) return e;
  if (int e = win::token_map(&m[5], V, s.B, s.N, s.Hkv, s.d, s.vs, 1, 32)) return e;
  if (int e = win::token_map(&m[6], dK, s.B, s.N, s.Hkv, s.d, kd, 1, 32)) return e;
  if (int e = win::token_map(&m[7], dV, s.B, s.N, s.Hkv, s.d, kd, 1, 32)) return e;
  if (int e = win::token_map(&m[8], O, s.B, s.Nq, s.Hq, s.d, hd, a.P, a.tok)) return e;
  return s.d == 128 ? bwd_launch<128>(a, m, st) : bwd_launch<64>(a, m, st);
}

}  // namespace pisa
