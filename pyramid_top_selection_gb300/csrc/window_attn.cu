// Sliding-window attention with sinks, forward: one warp per (query, head) row, keys in order
// with the running maximum and sum of the softmax.
#include "device.cuh"
#include "profile.h"
#include "window.h"

namespace pisa {

namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) window_fwd_kernel(const WinDims s, const __nv_bfloat16* Q,
                                                                 const __nv_bfloat16* K, const __nv_bfloat16* V,
                                                                 const int32_t* len, __nv_bfloat16* O, float* lse) {
  constexpr int E = D / 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(s.B) * s.Nq * s.Hq) return;
  const int lane = threadIdx.x & 31, h = static_cast<int>(row % s.Hq);
  const int64_t tok = row / s.Hq;
  const int i = static_cast<int>(tok % s.Nq), b = static_cast<int>(tok / s.Nq), kv = h / s.G;
  const int L = len ? max(0, min(len[b], s.N)) : s.N, p = i + s.off;
  float q[E], o[E] = {}, m = neg_inf(), l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(Q[tok * s.qs + h * D + lane * E + e]) * s.scale;
  if (p < L) {
    const int lo = max(0, p - s.window + 1);
    auto key = [&](int j) {
      const int64_t kr = static_cast<int64_t>(b) * s.N + j;
      float x = 0.f;
      for (int e = 0; e < E; ++e) x += q[e] * __bfloat162float(K[kr * s.ks + kv * D + lane * E + e]);
      x = warp_sum(x);
      const float mn = fmaxf(m, x), c = __expf(m - mn), w = __expf(x - mn);
      l = l * c + w;
      for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * __bfloat162float(V[kr * s.vs + kv * D + lane * E + e]);
      m = mn;
    };
    for (int j = 0; j < min(s.sinks, lo); ++j) key(j);
    for (int j = lo; j <= p; ++j) key(j);
  }
  for (int e = 0; e < E; ++e) O[row * D + lane * E + e] = __float2bfloat16_rn(l > 0.f ? o[e] / l : 0.f);
  if (lane == 0) lse[(static_cast<int64_t>(b) * s.Hq + h) * s.Nq + i] = l > 0.f ? m + logf(l) : neg_inf();
}

}  // namespace

int launch_window_fwd(const WinDims& s, const void* Q, const void* K, const void* V, const int32_t* len, void* O,
                      float* lse, char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(s.B) * s.Nq * s.Hq;
  const unsigned blocks = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
  auto k = s.d == 128 ? window_fwd_kernel<128> : window_fwd_kernel<64>;
  ProfScope ps(st, "window_fwd");
  k<<<blocks, 32 * kWarps, 0, st>>>(s, static_cast<const __nv_bfloat16*>(Q), static_cast<const __nv_bfloat16*>(K),
                                    static_cast<const __nv_bfloat16*>(V), len, static_cast<__nv_bfloat16*>(O), lse);
  return cudaGetLastError();
}

}  // namespace pisa
