// Sliding-window attention with sinks, forward: launches of window_fwd.cuh's kernel.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "profile.h"
#include "tmap.h"
#include "window_fwd.cuh"

namespace pisa {

namespace {

// The cluster launch of `splits` CTAs an item.
struct ClusterLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  ClusterLaunch(int grid, int splits, int smem, cudaStream_t st) {
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kFwdThreads);
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
  return ready(window_fwd_kernel<D, SPLIT, win::kWindow>, FwdSmem<D>::bytes, 168, SPLIT);
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
      if (cudaOccupancyMaxActiveClusters(&at_once, window_fwd_kernel<D, true, win::kWindow>, &c.cfg) != cudaSuccess) {
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
    return cudaLaunchKernelEx(&c.cfg, window_fwd_kernel<D, true, win::kWindow>, a, m[0], m[1], m[2], m[3], m[4], m[5]);
  }
  if (int e = fwd_ready<D, false>()) return e;
  window_fwd_kernel<D, false, win::kWindow><<<std::min(a.n_items, sm_count()), kFwdThreads, FwdSmem<D>::bytes, st>>>(a, m[0], m[1], m[2], m[3],
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
