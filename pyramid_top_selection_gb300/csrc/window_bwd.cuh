// Attention of rows over a run of keys each, backward, on the fifth-generation tensor cores: a sliding window with sinks
// (window_bwd.cu), or documents (doc_bwd.cuh).
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
#pragma once

#include <algorithm>

#include "device.cuh"
#include "internal.h"
#include "masks.cuh"
#include "pairs.cuh"

namespace pisa {

namespace {

using bf16 = __nv_bfloat16;
// Warps: 4 NG softmax and output (NG threads a row, 128 / NG columns each), then MMA, loader, MMA (dQ), items (dQ).
// NG = 2 is the window's; scores that cost more than the products hide take NG = 4 (launches).
constexpr int bwd_threads(int NG) { return 32 * (4 * NG + 4); }
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
  win::DocRows docs;       // documents (MASK), and what their gradients come from
  const bf16 *Q, *K, *V, *dO;
};

// One past the last valid token of sequence b, or of the documents.
template <int MASK>
__device__ __forceinline__ int end_of(const BwdArgs& a, int b) {
  return MASK == win::kWindow ? win::valid_len(a.len, b, a.s.N) : a.docs.bounds[a.s.N].y;
}

// COLS consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_cols(uint32_t taddr, float (&v)[64]) { tc::tmem_ld64(taddr, v); }
__device__ __forceinline__ void tmem_cols(uint32_t taddr, float (&v)[32]) { tc::tmem_ld32(taddr, v); }

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
template <int MASK>
__device__ __forceinline__ win::Item dq_item(const BwdArgs& a, int w) {
  const WinDims& s = a.s;
  const int tile = MASK == win::kWindow ? a.n_tiles - 1 - w / a.n_heads : a.docs.order[w / a.n_heads], hh = w % a.n_heads, set = hh % a.sets;
  win::Item it;
  it.b = hh / (s.Hkv * a.sets);
  it.kv = hh / a.sets % s.Hkv;
  it.h0 = it.kv * s.G + set * a.P;
  it.t0 = tile * a.tok;
  it.L = end_of<MASK>(a, it.b);
  if constexpr (MASK == win::kWindow) {
    const win::KeyList kl(s, it.L, s.off + it.t0, s.off + min(s.Nq, it.t0 + a.tok));
    it.lo = kl.lo;
    it.SP = kl.SP;
    it.n = (kl.n_cols + 127) >> 7;
  } else {
    const win::DocRange<MASK> r(a.docs, it.t0, min(s.Nq, it.t0 + a.tok));
    it.lo = r.lo;
    it.SP = 0;
    it.n = r.hi < r.lo ? 0 : (r.hi - r.lo + 128) >> 7;
  }
  it.first[0] = (it.b * s.Hkv + it.kv) * a.sets + set;
  it.first[1] = it.last[0] = it.last[1] = 0;
  return it;
}

// Documents: the rows of an item once more, those that keys which they do not see have made NaN (whole CTA).
template <int D, int MASK, int WARPS>
__device__ __forceinline__ void restore_dq(const BwdArgs& a, const win::Item& it) {
  const WinDims& s = a.s;
  const int lane = threadIdx.x & 31;
  const bf16 *K = a.K + it.kv * D, *V = a.V + it.kv * D;
  const int end_key = min(it.lo + 128 * it.n, it.L);
#pragma unroll 1
  for (int r = threadIdx.x >> 5; r < 128; r += WARPS) {
    const int i = it.t0 + (r >> a.lp), h = it.h0 + (r & (a.P - 1));
    if (i >= s.Nq) return;
    const int64_t row = static_cast<int64_t>(i) * s.Hq + h;
    if (!win::RowSum<D>::bad(a.dQ + row * D)) continue;
    const win::DocSpan<MASK> span(a.docs, i);
    const float lse = a.lse[static_cast<int64_t>(h) * s.Nq + i];
    float dl = 0.f;
    if (span.hi >= span.lo) {                                // else a row of zeros
      dl = a.delta[(static_cast<int64_t>(it.first[0]) * a.Nqp + it.t0) * a.P + r];
      if (!isfinite(lse) || !isfinite(dl)) continue;         // it is what its own values make it
      if (!win::rows_not_finite<D>(K, s.ks, it.lo, min(span.lo, end_key)) &&
          !win::rows_not_finite<D>(K, s.ks, max(it.lo, span.hi + 1), end_key))
        continue;
    }
    const bf16 *q = a.Q + i * s.qs + h * D, *g = a.dO + row * D;
    const float slope = MASK & win::kBias ? __ldg(a.docs.slopes + h) * kLog2e : 0.f;
    win::RowSum<D> o;
#pragma unroll 1
    for (int j0 = span.lo; j0 <= span.hi; j0 += 32) {
      const int j = j0 + lane;
      float w = 0.f;
      if (j <= span.hi) {
        float back;
        const float y = win::pair_score<MASK>(win::row_product<D>(q, K + j * s.ks), s.scale, a.docs.cap, slope, i - j, back);
        w = tc::ex2(y - lse * kLog2e) * back * (win::row_product<D>(g, V + j * s.vs) - dl);
      }
      o.add(w, K + j0 * s.ks, s.ks, min(32, span.hi + 1 - j0));
    }
    o.store(a.dQ + row * D, s.scale);
  }
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
template <int D, int MASK, int NG>
__global__ void __launch_bounds__(bwd_threads(NG), 1)
window_dq_kernel(const BwdArgs a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap domap,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ CUtensorMap kmap32, const __grid_constant__ CUtensorMap vmap32,
                 const __grid_constant__ CUtensorMap omap) {
  using M = DqSmem<D>;
  constexpr int NS = 4 * NG, COLS = 128 / NG;
  extern __shared__ __align__(1024) unsigned char sm[];      // SW128 tiles first
  __shared__ __align__(8) uint64_t q_full, q_empty, k_full[M::NK], k_empty[M::NK], v_full[M::NV], v_empty[M::NV],
      s_full[2], dp_full[2], d_full, ds_full[2], dq_done[2], dq_last, dq_empty, drain[2], never;
  __shared__ win::ItemRing s_items;
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort, s_spoiled;         // s_spoiled: a row came out as it may not be (documents)
  __shared__ float s_sum[NG][128];           // D of the rows, a sum for each of their threads

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
    tc::bar_init(&d_full, 32 * NS);
    tc::bar_init(&ds_full[0], 32 * NS);
    tc::bar_init(&ds_full[1], 32 * NS);
    tc::bar_init(&dq_done[0], 1);
    tc::bar_init(&dq_done[1], 1);
    tc::bar_init(&dq_last, 1);
    tc::bar_init(&dq_empty, 32 * NS);
    tc::bar_init(&drain[0], 1);
    tc::bar_init(&drain[1], 1);
    win::ring_init(s_items, NS + 3);
    tc::bar_init(&never, 1);
    tc::fence_bar_init();
    s_abort = s_spoiled = 0;
    if (MASK == win::kWindow && blockIdx.x == 0) *a.status = 0;      // nothing else writes it before the next kernel
  }
  if (warp == 0) tc::tmem_alloc(&tmem_base, 512);
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  if (MASK != win::kWindow) win::grid_wait();                // before the next kernel may start: it reads the documents' rows, too
  if (tid == 0) win::launch_dependents();
  const uint32_t tm = tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return win::wait(bar, parity, &s_abort, a.wait_ns); };
  auto get = [&](int k) { return win::ring_get(s_items, k, &s_abort, a.wait_ns); };
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };

  if (warp == NS + 1) {
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
  } else if (warp == NS) {
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
  } else if (warp == NS + 2) {
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
          win::product_ts<D, COLS>(tm + 384, tm + 128 * (g & 1), dK + st * kStage, j > 0);
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
  } else if (warp == NS + 3) {
    // ------------------------------------------------------------------ items, decoded ahead of the other
    // roles; their rows' lse is asked into L2 meanwhile
    const int rounds = win::rounds_of(a.n_items);
    for (int k = 0; k <= rounds; ++k) {
      const int64_t w = k < rounds ? win::item_of(k, a.n_items) : -1;
      win::Item it{};
      if (w >= 0) it = dq_item<MASK>(a, static_cast<int>(w));
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
  } else {
    // ------------------------------------------------------------------ softmax: row r, columns COLS g ..
    const int g = warp >> 2, r = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c1 = s.scale * kLog2e;
    constexpr bool CAP = MASK & win::kCap, BIAS = MASK & win::kBias;
    const win::Scores<CAP> scores(s.scale, CAP ? a.docs.cap : 0.f);
    win::Distance dist;
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
      win::DocSpan<MASK> span;
      if (MASK != win::kWindow && i < s.Nq) span = win::DocSpan<MASK>(a.docs, i);
      if (BIAS) dist.set(__ldg(a.docs.slopes + h) * kLog2e, span.hi > p);
      // x = P (through: times what a gradient takes through the cap), y = dP of key tile j; see: the visible columns,
      // where some are not
      auto load = [&](int j, float (&x)[COLS], float (&y)[COLS], uint32_t (&see)[COLS / 32], bool& masked, bool through) -> bool {
        const int k = n_k + j, v0 = 128 * j + COLS * g;
        bool ok = wait(&s_full[k & 1], (k >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc::after_sync();
        tmem_cols(tm + 128 * (k & 1) + COLS * g + lane_off, x);
        const int kb = kl.lo + v0 - kl.SP;
        int hi = row ? p - kb : -1, lo = max(p - s.window + 1, kl.lo) - kb, sk = s.sinks - v0;
        if constexpr (MASK != win::kWindow) {
          hi = span.hi - kb;
          lo = span.lo - kb;
          sk = 0;
        }
#pragma unroll
        for (int q = 0; q < COLS / 32; ++q) see[q] = 0xffffffffu;
        masked = !__all_sync(0xffffffffu, hi >= COLS - 1 && (lo <= 0 || sk >= COLS));
        if (masked) {
#pragma unroll
          for (int q = 0; q < COLS / 32; ++q)
            see[q] = win::bit_range(0, hi - 32 * q) & (win::bit_range(lo - 32 * q, 31) | win::bit_range(0, sk - 1 - 32 * q));
        }
        if constexpr (CAP || BIAS) {
          scores.apply(x);
          const float d0 = static_cast<float>(p - kb);
#pragma unroll
          for (int q = 0; q < COLS / 16; ++q) {
            const float b = nl + (BIAS && !dist.ahead ? dist.base(d0, 16 * q) : 0.f);
            const uint64_t bb = tc::pack2(b, b);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float& x0 = x[16 * q + 2 * c];
              float& x1 = x[16 * q + 2 * c + 1];
              const uint64_t y = tc::pack2(x0, x1);
              uint64_t z = tc::add2(y, bb);
              if (BIAS) {
                if (!dist.ahead) {
                  z = tc::add2(z, dist.part[c]);
                } else {
                  const float e0 = fabsf(d0 - static_cast<float>(16 * q + 2 * c)), e1 = fabsf(d0 - static_cast<float>(16 * q + 2 * c + 1));
                  z = tc::fma2(tc::pack2(e0, e1), tc::pack2(-dist.slope, -dist.slope), z);
                }
              }
              tc::unpack2(z, x0, x1);
              x0 = tc::ex2(x0);
              x1 = tc::ex2(x1);
              if (CAP && through) tc::unpack2(win::mul2(tc::pack2(x0, x1), scores.back(y)), x0, x1);
            }
          }
        } else {
          const uint64_t cc = tc::pack2(c1, c1), ll = tc::pack2(nl, nl);
#pragma unroll
          for (int c = 0; c < COLS; c += 2) {
            float y0, y1;
            tc::unpack2(tc::fma2(tc::pack2(x[c], x[c + 1]), cc, ll), y0, y1);
            x[c] = tc::ex2(y0);
            x[c + 1] = tc::ex2(y1);
          }
        }
        ok = wait(&dp_full[k & 1], (k >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc::after_sync();
        tmem_cols(tm + (n == 2 && j == 1 ? 384 : 256) + COLS * g + lane_off, y);
        return true;
      };
      float x[COLS], y[COLS];
      uint32_t see[COLS / 32];
      bool masked;
      // D: the sum of P dP, or dO . O of the tiles in shared memory
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      if (n <= 2) {
        for (int j = 0; ok && j < n; ++j) {
          ok = load(j, x, y, see, masked, false);
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < COLS; ++c)
            if (!masked || (see[c >> 5] >> (c & 31)) & 1) sum[c & 3] = fmaf(x[c], y[c], sum[c & 3]);
        }
        if (!ok) break;
      } else {
        ok = wait(&q_full, n_q & 1) && wait(&k_full[kk % M::NK], (kk / M::NK) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        uint64_t acc[2] = {0, 0};
        const unsigned char* po = sm + M::oK + kk % M::NK * M::TILE + r * 128;
        const unsigned char* pd = sm + M::oO + r * 128;
        constexpr int HC = D / 8 / NG;                       // 16-byte pieces of a thread's part of a row
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
      float dl = s_sum[0][r] + s_sum[1][r];
      if (NG == 4) dl += s_sum[NG - 2][r] + s_sum[NG - 1][r];
      if (n > 2 && tid == 0) tc::bar_arrive(&k_empty[kk % M::NK]);
      kk += n > 2;
      if (g == 0 && row) {
        const int64_t at = (static_cast<int64_t>(it.first[0]) * a.Nqp + it.t0) * a.P + r;
        a.nlse[at] = nl;
        a.delta[at] = dl;
      }
      for (int j = 0; j < n; ++j) {
        ok = load(j, x, y, see, masked, true);
        if (!ok) break;
        const int k = n_k + j;
        const uint32_t tS = tm + 128 * (k & 1) + COLS * g + lane_off;
        const uint64_t dd = tc::pack2(-dl, -dl);
#pragma unroll
        for (int c = 0; c < COLS; c += 2)
          tc::unpack2(win::mul2(tc::pack2(x[c], x[c + 1]), tc::add2(tc::pack2(y[c], y[c + 1]), dd)), x[c], x[c + 1]);
        if (masked) {
#pragma unroll
          for (int c = 0; c < COLS; ++c) x[c] = (see[c >> 5] >> (c & 31)) & 1 ? x[c] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < COLS / 32; ++q) {
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
      // dQ of the item, scaled: row r's 32 columns in turn for its threads (shared memory is full, and Q's and dO's tiles
      // already take the next item's, so the rows go out from registers)
      ok = wait(&dq_last, n_q & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::after_sync();
      ++n_q;
      const int64_t row0 = ((static_cast<int64_t>(it.b) * s.Nq + it.t0) * s.Hq + it.h0) * D + 8 * (lane & 3);
      win::Watch out;
#pragma unroll 1
      for (int q = g; q < D / 32; q += NG) {
        float y[32];
        tc::tmem_ld32(tm + 384 + 32 * q + lane_off, y);
        if (MASK != win::kWindow) out.add(y);
        uint32_t u[4][4];                                    // four 16-byte pieces of row r
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) u[c][k] = pack_bf16(s.scale * y[8 * c + 2 * k], s.scale * y[8 * c + 2 * k + 1]);
        win::transpose4(u, lane);                            // piece lane & 3 of four rows: 64 bytes of a row a store
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int rr = (r & ~3) + c;
          if (it.t0 + (rr >> a.lp) < s.Nq)
            *reinterpret_cast<uint4*>(a.dQ + row0 + (static_cast<int64_t>(rr >> a.lp) * s.Hq + (rr & (a.P - 1))) * D + 32 * q) =
                make_uint4(u[c][0], u[c][1], u[c][2], u[c][3]);
        }
      }
      tc::before_sync();
      tc::bar_arrive(&dq_empty);
      if (MASK != win::kWindow && out.bad()) s_spoiled = 1;
    }
    if (aborted() && g == 0) {                               // the rows of the item at hand and of those left
      for (; k_item < win::rounds_of(a.n_items); ++k_item) {
        const int64_t w = win::item_of(k_item, a.n_items);
        if (w < 0) break;
        const win::Item it = dq_item<MASK>(a, static_cast<int>(w));
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
      const win::Item it = dq_item<MASK>(a, static_cast<int>(w));
      if (tid < 128 && it.t0 + (tid >> a.lp) < s.Nq)
        a.nlse[(static_cast<int64_t>(it.first[0]) * a.Nqp + it.t0) * a.P + tid] = __int_as_float(0x7fc00000);
    }
  } else if (MASK != win::kWindow && s_spoiled) {
    for (int k = 0; k < win::rounds_of(a.n_items); ++k) {
      const int64_t w = win::item_of(k, a.n_items);
      if (w < 0) break;
      restore_dq<D, MASK, NS + 4>(a, dq_item<MASK>(a, static_cast<int>(w)));
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
  static constexpr int bytes = oBar + 512;           // d = 128: 231,936 of the 232,448 there are
};

struct DkvBars {
  uint64_t kv_full, q_full[3], q_empty[3], o_full[2], o_empty[2], st_full[2], st_empty[2], s_full, dp_full, p_full, ds_full,
      dv_done, dk_done, drain, never;
  uint32_t tmem_base;
  int abort, spoiled;              // spoiled: a row came out as it may not be (documents)
  float __align__(16) slope[64];   // the group's heads' slopes times -log2 e (kBias)
};
static_assert(sizeof(DkvBars) <= 512, "barrier block");

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
  // Documents: from the first token that sees the tile's first key to the last one of the last key's document.
  __device__ TokenRange(const win::DocRows& d, int T, int tok, int kt) {
    const int kb = 128 * kt;
    const int4 a = d.bounds[kb], z = d.bounds[min(kb + 127, T - 1)];
    const int first = kb >= a.x && kb < a.y && kb >= a.z ? kb : a.x, last = z.y;
    i0 = first & ~3;
    n = last > first ? (last - i0 + tok - 1) / tok : 0;
  }
};

template <int MASK>
__device__ __forceinline__ TokenRange tokens_of(const BwdArgs& a, int L, int kt) {
  if constexpr (MASK == win::kWindow) return TokenRange(a.s, a.tok, L, kt);
  else return TokenRange(a.docs, a.s.N, a.tok, kt);
}
// The token tiles of chunk c of nc: ct each, and all that are left in the last one (documents may be longer than was said).
__device__ __forceinline__ int chunk_tiles(int n, int c, int ct, int nc) { return max(0, c + 1 == nc ? n - c * ct : min(ct, n - c * ct)); }

struct DkvItem {
  int b, kv, kt, c, ct;            // chunk c, of ct token tiles, of the key tile's
  int64_t slot;                    // partial sums' slot, -1: the only chunk, written as it is
  // order: the key tiles' (NULL: as they come)
  __device__ DkvItem(const BwdArgs& a, int w, const int32_t* order) {
    const bool sink = w < a.n_snk;
    const int x = sink ? w : w - a.n_snk, tiles = sink ? a.n_st : a.n_kt - a.n_st;
    const int bh = x % a.n_bh;
    kt = x / a.n_bh % tiles + (sink ? 0 : a.n_st);
    if (order) kt = order[kt];
    c = x / a.n_bh / tiles;
    b = bh / a.s.Hkv;
    kv = bh % a.s.Hkv;
    ct = run_of(a, kt);
    slot = (sink ? a.ncs : a.nck) == 1 ? -1 : slot_of(a, kt, bh, c);
  }
  static __device__ int run_of(const BwdArgs& a, int kt) { return kt < a.n_st ? a.cts : a.ct; }
  // slots: sink tiles first ([kt][bh][ncs], where these are cut), then the others ([kt][bh][nck])
  static __device__ int64_t slot_of(const BwdArgs& a, int kt, int bh, int c) {
    if (kt < a.n_st) return (static_cast<int64_t>(kt) * a.n_bh + bh) * a.ncs + c;
    return (a.ncs > 1 ? a.n_snk : 0) + (static_cast<int64_t>(kt - a.n_st) * a.n_bh + bh) * a.nck + c;
  }
};

// Documents: the keys of an item, whose rows are those of tokens [t0, t1), once more, those that rows which do not see them have
// made NaN (whole CTA).
template <int D, int MASK, int WARPS>
__device__ __forceinline__ void restore_dkv(const BwdArgs& a, const DkvItem& it, int t0, int t1) {
  const WinDims& s = a.s;
  const int lane = threadIdx.x & 31, h0 = it.kv * s.G;
  const int64_t gs = static_cast<int64_t>(s.Hq) * D;
#pragma unroll 1
  for (int r = threadIdx.x >> 5; r < 128; r += WARPS) {
    const int j = 128 * it.kt + r;
    if (j >= s.N) return;
    const int64_t row = static_cast<int64_t>(j) * s.Hkv + it.kv;
    float* part = a.part + (it.slot * 2 * 128 + r) * D;      // dV, then dK
    const bool split = it.slot >= 0;
    const bool bad = split ? win::RowSum<D>::bad(part) || win::RowSum<D>::bad(part + 128 * D)
                           : win::RowSum<D>::bad(a.dV + row * D) || win::RowSum<D>::bad(a.dK + row * D);
    if (!bad) continue;
    const win::DocSeen seen(a.docs, j, s.N);
    const int from = max(t0, seen.first), to = min(t1, seen.end);
    auto other = [&](int x0, int x1) {                       // what does not see it is not finite
#pragma unroll 1
      for (int h = h0; h < h0 + s.G; ++h)
        if (win::rows_not_finite<D>(a.Q + h * D, s.qs, x0, x1) || win::rows_not_finite<D>(a.dO + h * D, gs, x0, x1)) return true;
      return false;
    };
    if (!other(t0, min(from, t1)) && !other(max(t0, to), t1)) continue;
    const bf16 *k = a.K + j * s.ks + it.kv * D, *v = a.V + j * s.vs + it.kv * D;
    win::RowSum<D> dk, dv;
#pragma unroll 1
    for (int h = h0; h < h0 + s.G; ++h) {
      const float slope = MASK & win::kBias ? __ldg(a.docs.slopes + h) * kLog2e : 0.f;
      const bf16 *Q = a.Q + h * D, *g = a.dO + h * D;
      const int64_t at = (static_cast<int64_t>(it.kv) * a.sets + (h - h0) / a.P) * a.Nqp;
#pragma unroll 1
      for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        float p = 0.f, ds = 0.f;
        if (i < to) {
          const int64_t x = (at + i) * a.P + (h - h0) % a.P;
          float back;
          const float y = win::pair_score<MASK>(win::row_product<D>(Q + i * s.qs, k), s.scale, a.docs.cap, slope, i - j, back);
          p = tc::ex2(y + a.nlse[x]);
          ds = p * back * (win::row_product<D>(g + i * gs, v) - a.delta[x]);
        }
        const int n = min(32, to - i0);
        dv.add(p, g + i0 * gs, gs, n);
        dk.add(ds, Q + i0 * s.qs, s.qs, n);
      }
    }
    if (split) {
      dv.store(part, 1.f);
      dk.store(part + 128 * D, s.scale);
    } else {
      dv.store(a.dV + row * D, 1.f);
      dk.store(a.dK + row * D, s.scale);
    }
  }
}

// One CTA per item: a tile of 128 keys of one KV head and a run of the row tiles that see it. TMEM:
// S^T (keys x rows; P^T in its place) at 0, dP^T (dS^T) at 128, dV at 256, dK at 256 + d. Per row
// tile n the MMA warp issues dV(n), S^T(n + 1), dK(n), dP^T(n + 1): the exponentials of one tile
// run under the dK and dP^T products, its dS under the next tile's dV and S^T. Each wait for a product
// that the next one overwrites the operand of is seen some 300 cycles after its issue; dK and dP^T a
// tile later would close these gaps, but hold two tiles' P in registers and spill (twice the time).
// 4 x 16384 rows of 16 heads over 4, a window of 1024, 4 sinks: 829 us, 1.29 PFLOP/s of its four products.
template <int D, int MASK, int NG>
__global__ void __launch_bounds__(bwd_threads(NG), 1)
window_dkv_kernel(const BwdArgs a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap domap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap dkmap, const __grid_constant__ CUtensorMap dvmap, int dq_ctas) {
  using M = DkvSmem<D>;
  constexpr int NS = 4 * NG, COLS = 128 / NG;
  extern __shared__ __align__(1024) unsigned char sm[];      // the only shared memory: SW128 tiles first
  DkvBars& bar = *reinterpret_cast<DkvBars*>(sm + M::oBar);
  auto &kv_full = bar.kv_full, &s_full = bar.s_full, &dp_full = bar.dp_full, &p_full = bar.p_full, &ds_full = bar.ds_full,
       &dv_done = bar.dv_done, &dk_done = bar.dk_done, &drain = bar.drain,
       &never = bar.never;
  auto &q_full = bar.q_full, &q_empty = bar.q_empty;
  auto &o_full = bar.o_full, &o_empty = bar.o_empty, &st_full = bar.st_full, &st_empty = bar.st_empty;
  uint32_t& tmem_base = bar.tmem_base;
  int &s_abort = bar.abort, &s_spoiled = bar.spoiled;

  const WinDims& s = a.s;
  const int tid = threadIdx.x, warp = win::uniform(tid >> 5), lane = tid & 31;
  const uint32_t aK = tc::su32(sm + M::oK), aV = tc::su32(sm + M::oV), aQ = tc::su32(sm + M::oQ), aO = tc::su32(sm + M::oO);

  const DkvItem it(a, blockIdx.x, MASK == win::kWindow ? nullptr : a.docs.key_order);
  const int kb = 128 * it.kt, L = end_of<MASK>(a, it.b);
  const int begin = MASK == win::kWindow ? 0 : a.docs.bounds[s.N].x;     // the first document's first token
  const TokenRange tr = tokens_of<MASK>(a, L, it.kt);
  // this chunk's row tiles: token tile n / sets, head set n % sets
  const int tile0 = it.c * it.ct, own = MASK == win::kWindow ? max(0, min(it.ct, tr.n - tile0)) : chunk_tiles(tr.n, it.c, it.ct, a.nck);
  const int n = win::uniform(own * a.sets);
  // This kernel starts while dQ's ends: what that wrote (statistics, status) is read after grid_wait only,
  // and one warp here waits for it in any case.
  if (warp == NS + 3) {
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
  if (warp == NS + 1 && lane == 0) {        // the first loads run under the rest of the CTA's start
    tc::bar_init(&kv_full, 1);
    for (int k = 0; k < M::NQ; ++k) {
      tc::bar_init(&q_full[k], 1);
      tc::bar_init(&q_empty[k], 1);
    }
    for (int k = 0; k < M::NO; ++k) {
      tc::bar_init(&o_full[k], 1);
      tc::bar_init(&o_empty[k], 1);
      tc::bar_init(&st_full[k], 1);
      tc::bar_init(&st_empty[k], NS);
    }
    tc::bar_init(&s_full, 1);
    tc::bar_init(&dp_full, 1);
    tc::bar_init(&p_full, 32 * NS);
    tc::bar_init(&ds_full, 32 * NS);
    tc::bar_init(&dv_done, 1);
    tc::bar_init(&dk_done, 1);
    tc::bar_init(&drain, 1);
    tc::bar_init(&never, 1);
    tc::fence_bar_init();
    s_abort = s_spoiled = 0;
    if (MASK & win::kBias)
      for (int h = 0; h < s.G; ++h) bar.slope[h] = -kLog2e * __ldg(a.docs.slopes + it.kv * s.G + h);
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

  if (warp == NS + 1) {
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
  } else if (warp == NS) {
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
          win::product_ts<D, COLS>(tm + 256, tm, dOt + so * kStage, k > 0);
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
          win::product_ts<D, COLS>(tm + 256 + D, tm + 128, dQt + qk * kStage, k > 0);
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
  } else if (warp < NS) {
    // ------------------------------------------------------------------ softmax: key (lane) r, rows COLS g ..
    const int g = warp >> 2, r = tid & 127, key = kb + r;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c1 = s.scale * kLog2e;
    // positions that see this key: [see_first, see_end)
    int see_first = key;
    int64_t see_end = key >= L ? 0 : key < s.sinks ? L : min(static_cast<int64_t>(L), static_cast<int64_t>(key) + s.window);
    if constexpr (MASK != win::kWindow) {
      const win::DocSeen seen(a.docs, key, s.N);
      see_first = seen.first;
      see_end = seen.end;
    }
    constexpr bool CAP = MASK & win::kCap, BIAS = MASK & win::kBias;
    const win::Scores<CAP> scores(s.scale, CAP ? a.docs.cap : 0.f);
    bool ok = true;
    for (int k = 0; k < n; ++k) {
      const int sq = k % M::NQ, ss = k & 1, pt0 = s.off + tile_tok(k);
      ok = wait(&st_full[ss], (k >> 1) & 1) && wait(&s_full, k & 1);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::after_sync();
      float x[COLS];
      const uint32_t tS = tm + COLS * g + lane_off;
      tmem_cols(tS, x);
      // column c is a row at position pt0 + c / P: visible iff lo <= c <= hi
      const int lo = max(-1, min(128, see_first - pt0)) * a.P - COLS * g;
      const int hi = static_cast<int>(max(int64_t(0), min(int64_t(128), see_end - pt0))) * a.P - 1 - COLS * g;
      uint32_t see[COLS / 32];
      const bool masked = !__all_sync(0xffffffffu, lo <= 0 && hi >= COLS - 1);
#pragma unroll
      for (int q = 0; q < COLS / 32; ++q) see[q] = masked ? win::bit_range(lo - 32 * q, hi - 32 * q) : 0xffffffffu;
      const float4* nl = reinterpret_cast<const float4*>(sm + M::oStat + ss * 1024 + 4 * COLS * g);
      const float4* dl = reinterpret_cast<const float4*>(sm + M::oStat + ss * 1024 + 512 + 4 * COLS * g);
      // P as bf16 over S^T's first half
      auto put = [&](int q, const uint32_t (&u)[16]) { tc::tmem_st16(tS + 16 * q, u); };
      if constexpr (CAP || BIAS) {
        // P goes out, and stays here times what a gradient takes through the cap
        scores.apply(x);
        const float* sl = bar.slope + k % a.sets * a.P;      // column c of the tile: token c / P, head c % P
        float few[4], step[4];                               // P < 4: four columns' slopes, and their tokens'
        if (BIAS) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            few[y] = sl[y & (a.P - 1)];
            step[y] = static_cast<float>(y >> a.lp);
          }
        }
        const int d0 = pt0 - key;
#pragma unroll
        for (int q = 0; q < COLS / 32; ++q) {
          uint32_t u[16];
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            float* e = x + 32 * q + c;
            const float4 l4 = nl[8 * q + c / 4];
            const uint64_t y[2] = {tc::pack2(e[0], e[1]), tc::pack2(e[2], e[3])};
            uint64_t z[2];
#pragma unroll
            for (int w = 0; w < 2; ++w) z[w] = tc::add2(y[w], w ? tc::pack2(l4.z, l4.w) : tc::pack2(l4.x, l4.y));
            if (BIAS) {
              const int col = COLS * g + 32 * q + c;
              const float d = static_cast<float>(d0 + (col >> a.lp));
              if (a.P >= 4) {
                const float4 s4 = *reinterpret_cast<const float4*>(sl + (col & (a.P - 1)));
                const uint64_t dd = tc::pack2(fabsf(d), fabsf(d));
                z[0] = tc::fma2(tc::pack2(s4.x, s4.y), dd, z[0]);
                z[1] = tc::fma2(tc::pack2(s4.z, s4.w), dd, z[1]);
              } else {
                z[0] = tc::fma2(tc::pack2(few[0], few[1]), tc::pack2(fabsf(d + step[0]), fabsf(d + step[1])), z[0]);
                z[1] = tc::fma2(tc::pack2(few[2], few[3]), tc::pack2(fabsf(d + step[2]), fabsf(d + step[3])), z[1]);
              }
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              float P0, P1;
              tc::unpack2(z[w], P0, P1);
              P0 = tc::ex2(P0);
              P1 = tc::ex2(P1);
              if (masked) {
                P0 = (see[q] >> (c + 2 * w)) & 1 ? P0 : 0.f;
                P1 = (see[q] >> (c + 2 * w + 1)) & 1 ? P1 : 0.f;
              }
              u[c / 2 + w] = pack_bf16(P0, P1);
              if (CAP) tc::unpack2(win::mul2(tc::pack2(P0, P1), scores.back(y[w])), P0, P1);
              e[2 * w] = P0;
              e[2 * w + 1] = P1;
            }
          }
          put(q, u);
        }
      } else {
        const uint64_t cc = tc::pack2(c1, c1);
#pragma unroll
        for (int c = 0; c < COLS; c += 4) {
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
          for (int c = 0; c < COLS; ++c) x[c] = (see[c >> 5] >> (c & 31)) & 1 ? x[c] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < COLS / 32; ++q) {
          uint32_t u[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) u[c] = pack_bf16(x[32 * q + 2 * c], x[32 * q + 2 * c + 1]);
          put(q, u);
        }
      }
      // rows at positions >= len (documents: and those before the first one) become zero in both tiles once S^T and dP^T have read them: P and dS
      // are 0 there, and dV and dK must not meet what padding holds
      if (g < 2 && ((L < s.N && tile_end(k) > L) || (MASK != win::kWindow && pt0 < begin))) {
        ok = wait(&dp_full, k & 1);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        const int base = g ? M::oO + k % M::NO * M::TILE : M::oQ + sq * M::TILE;
        if (pt0 + (r >> a.lp) >= L || (MASK != win::kWindow && pt0 + (r >> a.lp) < begin))
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
      const uint32_t tD = tm + 128 + COLS * g + lane_off;
#pragma unroll
      for (int q = 0; q < COLS / 32; ++q) {
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
    // output of key r: the first half of the warps dV, the others dK (scaled); of NG / 2 threads each takes its columns
    constexpr int NH = NG / 2;
    const int which = g / NH, part = g % NH;
    const float f = which ? s.scale : 1.f;
    const uint32_t tA = tm + 256 + D * which + lane_off;
    const float nan = __int_as_float(0x7fc00000);
    win::Watch out;
    if (it.slot >= 0) {
      float* o = a.part + ((it.slot * 2 + which) * 128 + (r & ~3)) * D + 4 * (lane & 3);
#pragma unroll 1
      for (int q = part; q < D / 32; q += NH) {
        float x[32];
        if (ok) {
          tc::tmem_ld32(tA + 32 * q, x);
          if (MASK != win::kWindow) out.add(x);
        }
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
      if (key < s.N && part == 0) {
        uint4* o = reinterpret_cast<uint4*>((which ? a.dK : a.dV) + ((static_cast<int64_t>(it.b) * s.N + key) * s.Hkv + it.kv) * D);
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(v, v, v, v);
      }
    } else {                                                 // through V's and K's shared memory
      const int base = which ? M::oK : M::oV;
#pragma unroll 1
      for (int x2 = part; x2 < M::KB; x2 += NH) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[32];
          tc::tmem_ld32(tA + 64 * x2 + 32 * h, x);
          if (MASK != win::kWindow) out.add(x);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = pack_bf16(f * x[8 * c + 2 * k], f * x[8 * c + 2 * k + 1]);
            *reinterpret_cast<uint4*>(sm + base + x2 * (128 * 128) + tc::sw128(r, 32 * h + 8 * c)) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          const int k0 = kb + 32 * (warp & 3);
          if (k0 < s.N)
            win::tma_store4(which ? &dkmap : &dvmap, 64 * x2, it.kv, k0, it.b,
                            tc::su32(sm + base) + x2 * (128 * 128) + (warp & 3) * (32 * 128));
          tc::bulk_commit();
        }
      }
      if (lane == 0) tc::bulk_wait<0>();
    }
    if (MASK != win::kWindow && out.bad()) s_spoiled = 1;
  }
  tc::before_sync();
  __syncthreads();
  if (tid == 0 && s_abort) {
    win::grid_wait();
    atomicOr(a.status, PISA_STATUS_TIMEOUT);
  }
  if (MASK != win::kWindow && s_spoiled && !s_abort) {
    win::fence_async_global();                               // dK and dV may have gone out by TMA
    win::grid_wait();
    restore_dkv<D, MASK, NS + 4>(a, it, max(begin, tile_tok(0)), min(L, tile_tok(n - 1) + a.tok));
  }
  if (warp == 0) {
    tc::after_sync();
    tc::tmem_free(tm, 512);
  }
}

// dK, dV of the key tiles that were cut into chunks: the chunks' partial sums in order.
// grid: (tiles x b kv, D / 4); a thread sums 4 elements.
template <int D, int MASK>
__global__ void __launch_bounds__(256) window_dkv_sum_kernel(const BwdArgs a, int first_kt) {
  const WinDims& s = a.s;
  const int kt = first_kt + blockIdx.x / a.n_bh, bh = blockIdx.x % a.n_bh, b = bh / s.Hkv, kv = bh % s.Hkv;
  const int L = end_of<MASK>(a, b);
  const TokenRange tr = tokens_of<MASK>(a, L, kt);
  const int ct = DkvItem::run_of(a, kt), all = (tr.n + ct - 1) / ct, chunks = MASK == win::kWindow ? all : min(all, a.nck);
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
inline void plan(BwdArgs& a) {
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

inline int64_t part_slots(const BwdArgs& a) {
  const int64_t sink = a.ncs > 1 ? a.n_snk : 0;
  const int64_t rest = a.nck > 1 ? static_cast<int64_t>(a.n_kt - a.n_st) * a.n_bh * a.nck : 0;
  return sink + rest;
}

}  // namespace
}  // namespace pisa
