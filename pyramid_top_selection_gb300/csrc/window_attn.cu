// Sliding-window attention with sinks, forward, on the fifth-generation tensor cores.
//
// Per row: O = softmax over the visible keys of (s q.k) times V, in one pass over the keys with the
// running maximum and sum of the softmax. P = 2^(c s_j - m) with c = scale log2 e; m follows the
// running maximum only when that grows by more than 2^8 (P, its sum and O then stay within fp32
// and bf16 range, and O is rescaled rarely); lse = (m + log2 l) ln 2.
//
// Persistent, one CTA per SM; a work item is 256 rows of one KV head: two 128-row tiles of (token,
// head) rows, P heads of the group together (window_tc.cuh), so the keys are read once for two tiles
// and the window's edges mask few columns. Items with the most keys come first. Roles:
//   * items (warp 10, one thread): decodes the CTA's items a few ahead, for all other roles;
//   * loader (warp 9, one lane issuing): Q tiles, then the item's key and value tiles of 128 columns
//     (KeyList: sinks and window as one list) by TMA into a ring of stages;
//   * MMA (warp 8, one lane issuing): per key tile and row tile, O += P V (P from tensor memory, V
//     as stored, MN-major), then the next S = Q K^T into the columns P has left. A tile's P V and
//     the next S alternate between the two row tiles, so one tile's softmax runs under the other's
//     products. (Two MMA warps, one a row tile, were slower, 1.76 against 1.59 ms at the 64K prefill:
//     their MMAs interleave one by one, and both products of a pair finish late.);
//   * softmax (warps 0-3 and 4-7, one row tile each, one row a thread): S row from tensor
//     memory into registers, masks where the tile touches an edge, maximum, exponentials, sum, P
//     as bf16 over the first half of S's columns; at the item's end O / l to bf16 through a
//     staging tile and TMA stores. In the tile that holds the sequence's end they also zero the
//     value rows at tokens >= len, so that padding's values (NaN, say) do not meet P = 0.
// TMEM: S (and P) of row tile t at 128 t, O at 256 + d t: all 512 columns at d = 128.
// P is rounded to bf16 for the product (2^-8 relative at most); the sum l takes it unrounded.
// Bound: the MMA warp, whose four groups of products a step are issued in some 2000 cycles and then
// waited for; the softmax is not (the time stays without any exponential). 65536 rows of 16 heads over 2, d =
// 128, a window of 4096: 1.48-1.52 ms a call in rows of calls, which run into the power limit (1.40-1.44 PFLOP/s,
// 73-75 % of a large library product's burst rate), 1.43 ms in a short burst (1.49 PFLOP/s). S in two halves,
// the upper one ahead of P's reading: 1.61 ms (64 columns cost 48 cycles a step of 16, 128 columns 64).
// With few rows (a short chunk against a long context) the items are fewer than the SMs. An item's key
// tiles are then cut into 2, 4, 8 or 16 runs, one CTA each, the CTAs a cluster: each lays its O, maxima
// and sums into its shared memory, and takes a share of the rows, which it reads from all of them and
// adds up in their order (no workspace, no second launch). The join takes some 3.5 us, as long as three key tiles.
// One token, 16 heads over 2 KV heads, 65536 keys: 68 us with 16 CTAs an item, 878 with one; 256 tokens
// of 8 heads and 4096 keys 20.0 (8 CTAs) and 57; 5 key tiles 12.4 (8), 14.2 (4), 14.6 (1).
// Every wait is bounded; one that gives up sets the CTA's abort flag, every role leaves, copies and
// MMAs in flight are drained, and the rows of the items left are poisoned.
#include <algorithm>
#include <atomic>

#include "device.cuh"
#include "internal.h"
#include "profile.h"
#include "tmap.h"
#include "window_tc.cuh"

namespace pisa {

namespace {

constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;                  // log2 growth of the maximum that O is rescaled for
constexpr uint64_t kDrainNs = 1000000000ull;   // bound of the drain waits (work already issued)
constexpr uint64_t kPatient = 1ull << 40;      // the item warp outwaits the others, whose giving up it sees

constexpr int kJoinTiles = 3;                  // the join of a split item in key tiles

template <int D>
struct FwdSmem {
  static constexpr int KB = D / 64;
  static constexpr int TILE = KB * 128 * 128;        // 128 rows x D bf16, SW128 blocks of 64 columns
  static constexpr int NST = 256 / D * 2;            // K / V stages: 128 KB in all
  static constexpr int oQ = 0, oKV = 2 * TILE, oStage = oKV + NST * TILE;
  static constexpr int STG = 32 * 128;               // a warp's 32 rows x 64 bf16
  static constexpr int bytes = oStage + 8 * STG;
};

struct FwdArgs {
  WinDims s;
  const int32_t* len;
  __nv_bfloat16* O;
  float* lse;
  int32_t* status;
  uint64_t wait_ns;
  int stall;
  int P, lp, tok;          // heads of a tile (P = 2^lp), tokens of a tile (128 / P)
  int n_tiles, n_heads, n_items;   // token tile pairs, (b, kv, head set) combinations
  int splits;              // CTAs of an item (SPLIT)
};

// Work item w: 2 x tok tokens of P heads.
__device__ __forceinline__ win::Item fwd_item(const FwdArgs& a, int w) {
  const WinDims& s = a.s;
  const int tile = a.n_tiles - 1 - w / a.n_heads, hh = w % a.n_heads, sets = s.G / a.P;
  win::Item it;
  it.b = hh / (s.Hkv * sets);
  it.kv = hh / sets % s.Hkv;
  it.h0 = it.kv * s.G + hh % sets * a.P;
  it.t0 = tile * 2 * a.tok;
  it.L = win::valid_len(a.len, it.b, s.N);
  const int p0 = s.off + it.t0, p1 = s.off + min(s.Nq, it.t0 + a.tok), p2 = s.off + min(s.Nq, it.t0 + 2 * a.tok);
  const win::KeyList kl(s, it.L, p0, p2);
  it.lo = kl.lo;
  it.SP = kl.SP;
  it.n = (kl.n_cols + 127) >> 7;
  const win::TileRange r0(s, kl, it.L, p0, p1), r1(s, kl, it.L, p0 + a.tok, p2);
  it.first[0] = r0.first;
  it.first[1] = r1.first;
  it.last[0] = r0.last;
  it.last[1] = r1.last;
  return it;
}

// SPLIT: one item per cluster of a.splits CTAs; otherwise a.splits is 1 and the CTAs are persistent.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
window_fwd_kernel(const FwdArgs a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap kmap32,
                  const __grid_constant__ CUtensorMap vmap32, const __grid_constant__ CUtensorMap omap) {
  using M = FwdSmem<D>;
  extern __shared__ __align__(1024) unsigned char sm[];      // SW128 tiles first
  __shared__ __align__(8) uint64_t q_full[2], q_empty[2], kv_full[M::NST], kv_empty[M::NST], s_full[2], p_full[2],
      pv_done[2], o_empty[2], drain, never;
  __shared__ win::ItemRing s_items;
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;

  const WinDims& s = a.s;
  const int tid = threadIdx.x, warp = win::uniform(tid >> 5), lane = tid & 31;
  const uint32_t aQ = tc::su32(sm + M::oQ), aKV = tc::su32(sm + M::oKV), aStage = tc::su32(sm + M::oStage);

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      tc::bar_init(&q_full[t], 1);
      tc::bar_init(&q_empty[t], 1);
      tc::bar_init(&s_full[t], 1);
      tc::bar_init(&p_full[t], 128);
      tc::bar_init(&pv_done[t], 1);
      tc::bar_init(&o_empty[t], 128);
    }
    for (int k = 0; k < M::NST; ++k) {
      tc::bar_init(&kv_full[k], 1);
      tc::bar_init(&kv_empty[k], 1);
    }
    win::ring_init(s_items, 10);
    tc::bar_init(&drain, 1);
    tc::bar_init(&never, 1);
    tc::fence_bar_init();
    s_abort = 0;
  }
  if (warp == 0) tc::tmem_alloc(&tmem_base, 512);
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  const uint32_t tm = tmem_base;
  const uint32_t dQ = win::desc_lo(aQ), dK = win::desc_lo(aKV), dV = win::desc_mn_lo(aKV, 128 * 128);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return win::wait(bar, parity, &s_abort, a.wait_ns); };
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };
  // positions of row tile t of an item: [p0, p1)
  auto tile_p0 = [&](const win::Item& it, int t) { return s.off + it.t0 + t * a.tok; };
  auto tile_p1 = [&](const win::Item& it, int t) { return s.off + min(s.Nq, it.t0 + (t + 1) * a.tok); };
  auto get = [&](int k) { return win::ring_get(s_items, k, &s_abort, a.wait_ns); };
  const int sink_tiles = (s.sinks + 127) >> 7;
  auto uses = [&](const win::Item& it, int t, int j) { return j <= it.last[t] && (j >= it.first[t] || j < sink_tiles); };
  // the CTA's key tiles [j0, j1) of an item
  const int rank = SPLIT ? static_cast<int>(win::cluster_rank()) : 0;
  auto run_begin = [&](const win::Item& it) { return SPLIT ? it.n * rank / a.splits : 0; };
  auto run_end = [&](const win::Item& it) { return SPLIT ? it.n * (rank + 1) / a.splits : it.n; };
  float m = neg_inf(), l = 0.f;                              // softmax threads: their row's maximum and sum
  int done = 0;                                              // key tiles that went into them

  if (warp >= 8) {
    win::regs_dec<88>();
    if (warp == 9) {
      // ---------------------------------------------------------------- loader
      int n_kv = 0, n_q[2] = {0, 0};           // loads issued
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const win::Item it = get(i);
        if (it.n < 0) break;
        const win::KeyList kl(it.lo, it.SP);
        auto load_q = [&](int t) -> bool {
          if (it.last[t] < 0) return true;
          if (!wait(&q_empty[t], (n_q[t] & 1) ^ 1)) return false;
          ++n_q[t];
          if (lane == 0) {
            tc::bar_expect_tx(&q_full[t], M::TILE);
#pragma unroll
            for (int kb = 0; kb < M::KB; ++kb)
              tc::tma_load4(aQ + t * M::TILE + kb * (128 * 128), &qmap, kb * 64, it.h0, it.t0 + t * a.tok, it.b, &q_full[t]);
          }
          __syncwarp();
          return true;
        };
        auto load_kv = [&](int v0, const CUtensorMap* big, const CUtensorMap* small) -> bool {
          const int st = n_kv % M::NST;
          if (!wait(&kv_empty[st], ((n_kv / M::NST) & 1) ^ 1)) return false;
          ++n_kv;
          if (lane == 0) {
            tc::bar_expect_tx(&kv_full[st], M::TILE);
            const uint32_t dst = aKV + st * M::TILE;
            if (v0 >= kl.SP) {
#pragma unroll
              for (int kb = 0; kb < M::KB; ++kb)
                tc::tma_load4(dst + kb * (128 * 128), big, kb * 64, it.kv, kl.key(v0), it.b, &kv_full[st]);
            } else {
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int kb = 0; kb < M::KB; ++kb)
                  tc::tma_load4(dst + kb * (128 * 128) + r * (32 * 128), small, kb * 64, it.kv, kl.key(v0 + 32 * r), it.b,
                                &kv_full[st]);
            }
          }
          __syncwarp();
          return true;
        };
        const int j0 = run_begin(it), j1 = run_end(it);
        if (j0 == j1) continue;
        ok = load_q(0) && load_kv(128 * j0, &kmap, &kmap32) && load_q(1) && load_kv(128 * j0, &vmap, &vmap32);
        for (int j = j0 + 1; ok && j < j1; ++j) ok = load_kv(128 * j, &kmap, &kmap32) && load_kv(128 * j, &vmap, &vmap32);
      }
      // whatever is still in flight lands before the CTA leaves
      for (int k = max(0, n_kv - M::NST); k < n_kv; ++k) tc::bar_wait(&kv_full[k % M::NST], (k / M::NST) & 1, kDrainNs);
      for (int t = 0; t < 2; ++t)
        if (n_q[t]) tc::bar_wait(&q_full[t], (n_q[t] - 1) & 1, kDrainNs);
    } else if (warp == 10) {
      // ---------------------------------------------------------------- items, decoded ahead of the other roles
      if (lane == 0) {
        const int rounds = SPLIT ? 1 : win::rounds_of(a.n_items);
        for (int k = 0; k <= rounds; ++k) {
          const int64_t w = k == rounds ? -1 : SPLIT ? blockIdx.x / a.splits : win::item_of(k, a.n_items);
          win::Item it{};
          if (w >= 0) it = fwd_item(a, static_cast<int>(w));
          else it.n = -1;                                    // only the last round can miss a CTA
          if (!win::ring_put(s_items, k, it, &s_abort, kPatient) || w < 0) break;
        }
      }
    } else if (warp == 8) {
      // ---------------------------------------------------------------- MMA (the warp together, one
      // lane issuing: operands stay in uniform registers)
      const bool leader = win::elect();
      int n_kv = 0;
      int n_q[2] = {0, 0}, n_p[2] = {0, 0}, n_o[2] = {0, 0};   // Q tiles, P V products, items of a row tile
      bool issued = false, ok = true;
      for (int i = 0; ok; ++i) {
        const win::Item it = get(i);
        if (it.n < 0) break;
        const int j0 = run_begin(it), j1 = run_end(it);
        if (j0 == j1) continue;
        if (a.stall && !wait(&never, 0)) { ok = false; break; }
        // key tile j is load n_kv + 2 (j - j0) of the ring, its values are the one after
        auto landed = [&](int k) { return wait(&kv_full[k % M::NST], (k / M::NST) & 1); };
        // S of row tile t from the key tile of load k; `last` of the row tile's, `free` the load's last use.
        // What S needs is waited for while the product before it still runs.
        auto issue_s = [&](int t, int k, bool last, bool free) -> bool {
          if (n_p[t] > 0 && !wait(&pv_done[t], (n_p[t] - 1) & 1)) return false;   // P has been read
          tc::after_sync();
          if (leader) {
            win::product_ss<D>(tm + 128 * t, dQ + t * (M::TILE >> 4), dK + k % M::NST * (M::TILE >> 4));
            tc::commit(&s_full[t]);
            if (free) tc::commit(&kv_empty[k % M::NST]);
            if (last) tc::commit(&q_empty[t]);
          }
          __syncwarp();
          return true;
        };
        auto issue_pv = [&](int t, int k, bool accumulate, bool free) -> bool {
          if (!accumulate && !wait(&o_empty[t], (n_o[t]++ & 1) ^ 1)) return false;   // the last item's O is out
          if (!wait(&p_full[t], n_p[t] & 1)) return false;
          tc::after_sync();
          if (leader) {
            win::product_ts<D, 128>(tm + 256 + D * t, tm + 128 * t, dV + k % M::NST * (M::TILE >> 4), accumulate);
            tc::commit(&pv_done[t]);
            if (free) tc::commit(&kv_empty[k % M::NST]);
          }
          __syncwarp();
          ++n_p[t];
          return true;
        };
        bool has0 = uses(it, 0, j0), has1 = uses(it, 1, j0), acc0 = false, acc1 = false;
        issued = true;
        ok = landed(n_kv) && (it.last[0] < 0 || wait(&q_full[0], n_q[0]++ & 1));
        if (ok && has0) ok = issue_s(0, n_kv, it.last[0] == j0, !has1);
        ok = ok && (it.last[1] < 0 || wait(&q_full[1], n_q[1]++ & 1));
        if (ok && has1) ok = issue_s(1, n_kv, it.last[1] == j0, true);
        ok = ok && landed(n_kv + 1);
        for (int j = j0; ok && j < j1; ++j) {
          const int k = n_kv + 2 * (j - j0) + 1;
          const bool more = !SPLIT || j + 1 < j1;            // (an item's last tile has no next one anyway)
          const bool next0 = more && uses(it, 0, j + 1), next1 = more && uses(it, 1, j + 1);
          if (has0 && !issue_pv(0, k, acc0, !has1)) { ok = false; break; }
          if (j + 1 < j1 && !landed(k + 1)) { ok = false; break; }
          if (next0 && !issue_s(0, k + 1, it.last[0] == j + 1, !next1)) { ok = false; break; }
          if (has1 && !issue_pv(1, k, acc1, true)) { ok = false; break; }
          if (j + 1 < j1 && !landed(k + 2)) { ok = false; break; }
          if (next1 && !issue_s(1, k + 1, it.last[1] == j + 1, true)) { ok = false; break; }
          acc0 |= has0;
          acc1 |= has1;
          has0 = next0;
          has1 = next1;
        }
        n_kv += 2 * (j1 - j0);
      }
      if (issued) {
        if (leader) tc::commit(&drain);
        __syncwarp();
        tc::bar_wait(&drain, 0, kDrainNs);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax, output
    win::regs_inc<208>();
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tm + 128 * t + lane_off, tO = tm + 256 + D * t + lane_off;
    const float c1 = s.scale * kLog2e;
    int n_s = 0, n_kv = 0;                     // key tiles done by this row tile; stages used by earlier items
    int i = 0;
    for (int n = 0;; ++i, n_kv += 2 * n) {
      const win::Item it = get(i);
      if (it.n < 0) break;
      const int j0 = run_begin(it), j1 = run_end(it);
      n = j1 - j0;
      const int L = it.L;
      const win::KeyList kl(it.lo, it.SP);
      const int p0 = tile_p0(it, t), p1 = tile_p1(it, t);
      const int j_first = t ? it.first[1] : it.first[0], j_last = t ? it.last[1] : it.last[0];
      const int p = p0 + (r >> a.lp), h = it.h0 + (r & (a.P - 1));
      const bool row = p < p1 && p < L;
      if (!SPLIT) {
        m = neg_inf();
        l = 0.f;
        done = 0;
      }
      bool ok = true;
      for (int j = j0; j < j1; ++j) {
        const int v0 = 128 * j;
        if (j > j_last || (j < j_first && j >= sink_tiles)) continue;
        ok = wait(&s_full[t], n_s & 1);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc::after_sync();
        float x[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y[32];
          tc::tmem_ld32(tS + 32 * q, y);
#pragma unroll
          for (int c = 0; c < 32; ++c) x[32 * q + c] = y[c];
        }
        // column c is key kb + c (or sink v0 + c): visible iff c <= hi and (c >= lo or c < sk)
        const int kb = kl.lo + v0 - kl.SP;
        const int hi = row ? p - kb : -1, lo = max(p - s.window + 1, kl.lo) - kb, sk = s.sinks - v0;
        const bool all = hi >= 127 && (lo <= 0 || sk >= 128);
        if (!__all_sync(0xffffffffu, all)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t see = win::bit_range(0, hi - 32 * q) & (win::bit_range(lo - 32 * q, 31) | win::bit_range(0, sk - 1 - 32 * q));
#pragma unroll
            for (int c = 0; c < 32; ++c) x[32 * q + c] = (see >> c) & 1 ? x[32 * q + c] : neg_inf();
          }
        }
        // P = 2^(c1 x - mm) over S's first half, its sum, the row's maximum
        uint64_t sum[2];
        const uint64_t cc = tc::pack2(c1, c1);
        auto exps = [&](float mm) {
          const uint64_t nm = tc::pack2(-mm, -mm);
          sum[0] = sum[1] = 0;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t u[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float y0, y1;
              tc::unpack2(tc::fma2(tc::pack2(x[16 * q + 2 * c], x[16 * q + 2 * c + 1]), cc, nm), y0, y1);
              y0 = tc::ex2(y0);
              y1 = tc::ex2(y1);
              sum[c & 1] = tc::add2(sum[c & 1], tc::pack2(y0, y1));
              u[c] = pack_bf16(y0, y1);
            }
            asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(tS + 8 * q), "r"(u[0]),
                         "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                         : "memory");
          }
        };
        auto row_max = [&]() {
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmaxf(x[q], x[4 + q]);
#pragma unroll
          for (int c = 8; c < 128; c += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = tc::max3(mx[q], x[c + q], x[c + 4 + q]);
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c1;
        };
        // After an item's first tile the exponentials do not wait for the tile's maximum: they are taken
        // against the maximum so far, and once more in the rare tile whose maximum outgrows it.
        float top;
        bool grow;
        if (done) {
          exps(m > neg_inf() ? m : 0.f);
          top = row_max();
          grow = top > m + kSlack;                           // also from m = -inf
        } else {
          top = row_max();
          grow = true;
        }
        if (__any_sync(0xffffffffu, grow)) {
          const bool fix = grow && m > neg_inf();            // something has been accumulated
          float f = 1.f;
          if (grow) {
            f = fix ? tc::ex2(m - top) : 1.f;
            m = top;
            l *= f;
          }
          if (__any_sync(0xffffffffu, fix)) {                // O waits for the product before, then follows
            ok = wait(&pv_done[t], (n_s - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc::after_sync();
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t u[16];
              win::tmem_ld16(tO + 16 * q, u);
#pragma unroll
              for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(__uint_as_float(u[c]) * f);
              tc::tmem_st16(tO + 16 * q, u);
            }
          }
          exps(m > neg_inf() ? m : 0.f);
        }
        // padding's values (only the last tile can reach past the sequence) become zero before this row
        // tile's product; the other row tile writes the same zeros before its own
        if (L < s.N && kl.key(v0 + 127) >= L) {
          const int k = n_kv + 2 * (j - j0) + 1, st = k % M::NST;
          ok = wait(&kv_full[st], (k / M::NST) & 1);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          if (v0 + r >= kl.SP && kl.key(v0 + r) >= L)
            for (int c = 0; c < M::KB * 8; ++c)
              *reinterpret_cast<uint4*>(sm + M::oKV + st * M::TILE + (c >> 3) * (128 * 128) + r * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          tc::fence_async_smem();
        }
        tc::tmem_wait_st();
        tc::before_sync();
        tc::bar_arrive(&p_full[t]);
        float s0, s1;
        tc::unpack2(tc::add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        ++n_s;
        ++done;
      }
      if (!ok) break;
      if (p0 >= s.off + s.Nq) continue;                      // a tile past the last query
      if (done) {
        ok = wait(&pv_done[t], (n_s - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc::after_sync();
      }
      if (SPLIT) continue;                                   // the cluster's results are joined below
      if (p < p1)
        a.lse[(static_cast<int64_t>(it.b) * s.Hq + h) * s.Nq + p - s.off] = l == 0.f ? neg_inf() : (m + log2f(l)) * kLn2;
      const float inv = 1.f / l;                             // l = 0: an empty row, whose output is 0
      unsigned char* stg = sm + M::oStage + warp * M::STG;
      const int tk = it.t0 + t * a.tok + ((warp & 3) * 32 >> a.lp);   // the warp's first token
#pragma unroll 1
      for (int kb = 0; kb < M::KB; ++kb) {
        uint32_t u[32];
        if (done) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float y[32];
            tc::tmem_ld32(tO + 64 * kb + 32 * q, y);
#pragma unroll
            for (int c = 0; c < 16; ++c) u[16 * q + c] = l == 0.f ? 0u : pack_bf16(y[2 * c] * inv, y[2 * c + 1] * inv);
          }
          if (kb == M::KB - 1) {
            tc::before_sync();
            tc::bar_arrive(&o_empty[t]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) u[c] = 0u;
        }
        if (lane == 0) tc::bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (tk < s.Nq) win::tma_store4(&omap, 64 * kb, it.h0, tk, it.b, aStage + warp * M::STG);
          tc::bulk_commit();
        }
      }
    }
    if (lane == 0) tc::bulk_wait<0>();
    if (!SPLIT && aborted()) {                               // the rows of the item at hand and of those left
      for (; i < win::rounds_of(a.n_items); ++i) {
        const int64_t w = win::item_of(i, a.n_items);
        if (w < 0) break;
        const win::Item it = fwd_item(a, static_cast<int>(w));
        const int row = it.t0 + t * a.tok + (r >> a.lp), h = it.h0 + (r & (a.P - 1));
        if (row >= s.Nq) continue;
        a.lse[(static_cast<int64_t>(it.b) * s.Hq + h) * s.Nq + row] = __int_as_float(0x7fc00000);
        uint4* o = reinterpret_cast<uint4*>(a.O + ((static_cast<int64_t>(it.b) * s.Nq + row) * s.Hq + h) * D);
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
      }
    }
  }
  if (SPLIT) {
    // ------------------------------------------------------------------ join: every CTA lays its O and (m, l)
    // into shared memory, over the key tiles that nothing reads any more, and takes 1 / splits of the rows
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    const win::Item it = fwd_item(a, blockIdx.x / a.splits);
    float* part = reinterpret_cast<float*>(sm + M::oKV);     // [256][D], a row's 16-byte pieces permuted by its number
    float2* stat = reinterpret_cast<float2*>(sm + M::oStage);   // [256] (m, l)
    constexpr int PC = D / 4;
    if (warp < 8) {
      stat[tid] = make_float2(m, l);
      if (done)
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t u[16];
          win::tmem_ld16(tm + 256 + D * (warp >> 2) + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 16 * q, u);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            reinterpret_cast<uint4*>(part)[tid * PC + ((4 * q + c) ^ (tid & (PC - 1)))] =
                make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
        }
    }
    __syncwarp();
    win::cluster_sync();
    if (warp < 8) {
      // a warp's 32 / splits rows x splits CTAs are 32 pairs: one a lane for the statistics, then all of
      // them (half of them, at d = 64) in turn for a lane's four columns, eight reads under way at a time
      const int n = a.splits, ln = __ffs(n) - 1, x0 = (rank * 8 + warp) * (32 >> ln);
      const float2 ml = win::ld_cluster_f2(stat + x0 + (lane >> ln), lane & (n - 1));
      const bool bad = __any_sync(0xffffffffu, win::ld_cluster_u32(&s_abort, lane & (n - 1)) != 0);
      float top = ml.x;
      for (int d = n >> 1; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      float f = ml.y == 0.f ? 0.f : tc::ex2(ml.x - top);     // (a row's NaN goes on)
      float sum = f * ml.y;
      for (int d = n >> 1; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      int64_t row = -1;                                      // (token, head) of the lane's pair
      {
        const int x = x0 + (lane >> ln), t = x >> 7, r = x & 127, p = tile_p0(it, t) + (r >> a.lp), h = it.h0 + (r & (a.P - 1));
        if (p < tile_p1(it, t)) {
          row = (it.b * static_cast<int64_t>(s.Nq) + p - s.off) * s.Hq + h;
          if ((lane & (n - 1)) == 0)
            a.lse[(static_cast<int64_t>(it.b) * s.Hq + h) * s.Nq + p - s.off] =
                bad ? __int_as_float(0x7fc00000) : sum == 0.f ? neg_inf() : (top + log2f(sum)) * kLn2;
        }
      }
      f *= bad ? __int_as_float(0x7fc00000) : sum == 0.f ? 0.f : 1.f / sum;
      constexpr int HALF = 32 / PC;                          // rows at a time
      const int pc = lane % PC, e0 = lane / PC * (32 / HALF);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int e = e0; e < e0 + 32 / HALF; e += 8) {
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int x = x0 + ((e + k) >> ln);
          const float fc = __shfl_sync(0xffffffffu, f, e + k);
          v[k] = make_float4(fc, fc, fc, fc);                // zeros: nothing seen there, perhaps nothing written
          if (fc != 0.f && !bad) v[k] = win::ld_cluster_f4(part + x * D + ((pc ^ (x & (PC - 1))) << 2), (e + k) & (n - 1));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float fc = __shfl_sync(0xffffffffu, f, e + k);
          const int64_t to = __shfl_sync(0xffffffffu, row, e + k);
          o.x += fc * v[k].x;
          o.y += fc * v[k].y;
          o.z += fc * v[k].z;
          o.w += fc * v[k].w;
          if (((e + k + 1) & (n - 1)) == 0) {                // the row's last CTA
            if (to >= 0) *reinterpret_cast<uint2*>(a.O + to * D + 4 * pc) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
            o = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
    }
    __syncwarp();
    win::cluster_sync();                                     // nobody leaves while its results are read
  }
  tc::before_sync();
  __syncthreads();
  if (tid == 0 && s_abort && a.status) atomicOr(a.status, PISA_STATUS_TIMEOUT);
  if (warp == 0) {
    tc::after_sync();
    tc::tmem_free(tm, 512);
  }
}

// The cluster launch of `splits` CTAs an item.
struct ClusterLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  ClusterLaunch(int grid, int splits, int smem, cudaStream_t st) {
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(splits);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  ClusterLaunch(const ClusterLaunch&) = delete;
};

// The softmax warps' larger register share is drawn from what the CTA was launched with: 168 a thread.
template <int D, bool SPLIT>
int fwd_ready() {
  static win::Ready ready;
  return ready(window_fwd_kernel<D, SPLIT>, FwdSmem<D>::bytes, 168, SPLIT);
}

// CTAs of an item, one of 1, 2, 4, 8, 16: the number with the fewest key tiles for the longest run,
// the join counted as kJoinTiles of them, among those whose clusters all run at one time.
template <int D>
int fwd_splits(int64_t items, int64_t tiles) {
  static std::atomic<int> known[64][5];                      // clusters of 2^k CTAs at one time + 1, per device
  int best = 1, dev = 0;
  if (items * 2 > sm_count() || tiles < kJoinTiles + 2) return 1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64 || fwd_ready<D, true>()) return 1;
  for (int k = 1; k <= 4; ++k) {
    const int n = 1 << k;
    if (items * n > sm_count()) break;
    const int64_t cost = (tiles + n - 1) / n + kJoinTiles, now = (tiles + best - 1) / best + (best > 1 ? kJoinTiles : 0);
    if (cost >= now) continue;
    int at_once = known[dev][k].load(std::memory_order_relaxed) - 1;
    if (at_once < 0) {
      ClusterLaunch c(n, n, FwdSmem<D>::bytes, nullptr);
      if (cudaOccupancyMaxActiveClusters(&at_once, window_fwd_kernel<D, true>, &c.cfg) != cudaSuccess) {
        cudaGetLastError();
        at_once = 0;
      }
      known[dev][k].store(at_once + 1, std::memory_order_relaxed);
    }
    if (items <= at_once) best = n;
  }
  return best;
}

template <int D>
int fwd_launch(FwdArgs& a, int64_t tiles, const CUtensorMap* m, cudaStream_t st) {
  a.splits = fwd_splits<D>(a.n_items, tiles);
  ProfScope ps(st, "window_fwd");
  if (a.splits > 1) {
    ClusterLaunch c(a.n_items * a.splits, a.splits, FwdSmem<D>::bytes, st);
    return cudaLaunchKernelEx(&c.cfg, window_fwd_kernel<D, true>, a, m[0], m[1], m[2], m[3], m[4], m[5]);
  }
  if (int e = fwd_ready<D, false>()) return e;
  window_fwd_kernel<D, false><<<std::min(a.n_items, sm_count()), kThreads, FwdSmem<D>::bytes, st>>>(a, m[0], m[1], m[2], m[3],
                                                                                                     m[4], m[5]);
  return cudaGetLastError();
}

}  // namespace

int launch_window_fwd(const WinDims& s, const void* Q, const void* K, const void* V, const int32_t* len, void* O,
                      float* lse, char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  FwdArgs a{};
  a.s = s;
  a.len = len;
  a.O = static_cast<__nv_bfloat16*>(O);
  a.lse = lse;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.wait_ns = wait_limit_ns();
  a.stall = test_stall();
  a.P = win::packed_heads(s.G);
  a.lp = win::log2_of(a.P);
  a.tok = 128 / a.P;
  a.n_tiles = (s.Nq + 2 * a.tok - 1) / (2 * a.tok);
  a.n_heads = s.B * s.Hkv * (s.G / a.P);
  const int64_t items = static_cast<int64_t>(a.n_tiles) * a.n_heads;   // < B N Hq
  a.n_items = static_cast<int>(items);
  CUtensorMap m[6];
  if (int e = win::token_map(&m[0], Q, s.B, s.Nq, s.Hq, s.d, s.qs, a.P, a.tok)) return e;
  if (int e = win::token_map(&m[1], K, s.B, s.N, s.Hkv, s.d, s.ks, 1, 128)) return e;
  if (int e = win::token_map(&m[2], V, s.B, s.N, s.Hkv, s.d, s.vs, 1, 128)) return e;
  m[3] = m[1];                     // the sinks' boxes, where there are any
  m[4] = m[2];
  if (s.sinks > 0) {
    if (int e = win::token_map(&m[3], K, s.B, s.N, s.Hkv, s.d, s.ks, 1, 32)) return e;
    if (int e = win::token_map(&m[4], V, s.B, s.N, s.Hkv, s.d, s.vs, 1, 32)) return e;
  }
  if (int e = win::token_map(&m[5], O, s.B, s.Nq, s.Hq, s.d, static_cast<int64_t>(s.Hq) * s.d, a.P, 32 / a.P)) return e;
  if (ws) {
    cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
    if (e != cudaSuccess) return e;
  }
  // key tiles of the longest item
  const int64_t cols = std::min<int64_t>(s.N, s.window + 2ll * a.tok - 1) + (s.sinks + 31) / 32 * 32;
  const int64_t tiles = (cols + 127) / 128;
  return s.d == 128 ? fwd_launch<128>(a, tiles, m, st) : fwd_launch<64>(a, tiles, m, st);
}

}  // namespace pisa
