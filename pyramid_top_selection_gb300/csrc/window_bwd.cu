// Sliding-window attention with sinks, backward: D = dO . O per row, then dQ with one warp per
// (query, head) row over its keys, and dK, dV with one warp per (key, KV head) over the rows
// that see it (no atomics: the order of every sum is fixed).
#include "device.cuh"
#include "profile.h"
#include "window.h"

namespace pisa {

size_t align256(size_t x);

namespace {

constexpr int kWarps = 8;
using bf16 = __nv_bfloat16;

struct WinBwdArgs {
  WinDims s;
  const bf16 *Q, *K, *V, *O, *dO;
  const float* lse;
  const int32_t* len;
  float* delta;    // [B, Nq, Hq]
  bf16 *dQ, *dK, *dV;
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps) window_dq_kernel(const WinBwdArgs a) {
  constexpr int E = D / 32;
  const WinDims& s = a.s;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(s.B) * s.Nq * s.Hq) return;
  const int lane = threadIdx.x & 31, h = static_cast<int>(row % s.Hq);
  const int64_t tok = row / s.Hq;
  const int i = static_cast<int>(tok % s.Nq), b = static_cast<int>(tok / s.Nq), kv = h / s.G;
  const int L = a.len ? max(0, min(a.len[b], s.N)) : s.N, p = i + s.off;
  float q[E], g[E], acc[E] = {}, dl = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.Q[tok * s.qs + h * D + lane * E + e]);
    g[e] = __bfloat162float(a.dO[row * D + lane * E + e]);
    dl += g[e] * __bfloat162float(a.O[row * D + lane * E + e]);
  }
  dl = warp_sum(dl);
  if (lane == 0) a.delta[row] = dl;
  if (p < L) {
    const float ls = a.lse[(static_cast<int64_t>(b) * s.Hq + h) * s.Nq + i];
    const int lo = max(0, p - s.window + 1);
    auto key = [&](int j) {
      const int64_t kr = static_cast<int64_t>(b) * s.N + j;
      float x = 0.f, y = 0.f, k[E];
      for (int e = 0; e < E; ++e) {
        k[e] = __bfloat162float(a.K[kr * s.ks + kv * D + lane * E + e]);
        x += q[e] * k[e];
        y += g[e] * __bfloat162float(a.V[kr * s.vs + kv * D + lane * E + e]);
      }
      const float ds = __expf(s.scale * warp_sum(x) - ls) * (warp_sum(y) - dl) * s.scale;
      for (int e = 0; e < E; ++e) acc[e] += ds * k[e];
    };
    for (int j = 0; j < min(s.sinks, lo); ++j) key(j);
    for (int j = lo; j <= p; ++j) key(j);
  }
  for (int e = 0; e < E; ++e) a.dQ[row * D + lane * E + e] = __float2bfloat16_rn(acc[e]);
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) window_dkv_kernel(const WinBwdArgs a) {
  constexpr int E = D / 32;
  const WinDims& s = a.s;
  const int64_t kr = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (kr >= static_cast<int64_t>(s.B) * s.N * s.Hkv) return;
  const int lane = threadIdx.x & 31, kv = static_cast<int>(kr % s.Hkv);
  const int64_t tok = kr / s.Hkv;
  const int j = static_cast<int>(tok % s.N), b = static_cast<int>(tok / s.N);
  const int L = a.len ? max(0, min(a.len[b], s.N)) : s.N;
  float dk[E] = {}, dv[E] = {};
  if (j < L) {
    float k[E], v[E];
    for (int e = 0; e < E; ++e) {
      k[e] = __bfloat162float(a.K[tok * s.ks + kv * D + lane * E + e]);
      v[e] = __bfloat162float(a.V[tok * s.vs + kv * D + lane * E + e]);
    }
    const int64_t hi = j < s.sinks ? L : min(static_cast<int64_t>(L), static_cast<int64_t>(j) + s.window);
    for (int p = max(j, s.off); p < hi; ++p)
      for (int h = kv * s.G; h < (kv + 1) * s.G; ++h) {
        const int64_t qt = static_cast<int64_t>(b) * s.Nq + p - s.off, row = qt * s.Hq + h;
        float q[E], g[E], x = 0.f, y = 0.f;
        for (int e = 0; e < E; ++e) {
          q[e] = __bfloat162float(a.Q[qt * s.qs + h * D + lane * E + e]);
          g[e] = __bfloat162float(a.dO[row * D + lane * E + e]);
          x += q[e] * k[e];
          y += g[e] * v[e];
        }
        const float w = __expf(s.scale * warp_sum(x) - a.lse[(static_cast<int64_t>(b) * s.Hq + h) * s.Nq + p - s.off]);
        const float ds = w * (warp_sum(y) - a.delta[row]) * s.scale;
        for (int e = 0; e < E; ++e) {
          dk[e] += ds * q[e];
          dv[e] += w * g[e];
        }
      }
  }
  for (int e = 0; e < E; ++e) {
    a.dK[kr * D + lane * E + e] = __float2bfloat16_rn(dk[e]);
    a.dV[kr * D + lane * E + e] = __float2bfloat16_rn(dv[e]);
  }
}

}  // namespace

WinBwdWs window_bwd_ws(const WinDims& s) {
  WinBwdWs w{};
  w.status = 0;
  w.delta = 256;
  w.total = w.delta + align256(static_cast<size_t>(s.B) * s.Nq * s.Hq * 4);
  return w;
}

int launch_window_bwd(const WinDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                      const void* dO, const int32_t* len, void* dQ, void* dK, void* dV, char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return e;
  auto c = [](const void* p) { return static_cast<const bf16*>(p); };
  auto m = [](void* p) { return static_cast<bf16*>(p); };
  const WinBwdArgs a{s, c(Q), c(K), c(V), c(O), c(dO), lse, len,
                     reinterpret_cast<float*>(ws + window_bwd_ws(s).delta), m(dQ), m(dK), m(dV)};
  const int64_t rows = static_cast<int64_t>(s.B) * s.Nq * s.Hq, keys = static_cast<int64_t>(s.B) * s.N * s.Hkv;
  {
    ProfScope ps(st, "window_dq");
    (s.d == 128 ? window_dq_kernel<128> : window_dq_kernel<64>)
        <<<static_cast<unsigned>((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ProfScope ps(st, "window_dkv");
  (s.d == 128 ? window_dkv_kernel<128> : window_dkv_kernel<64>)
      <<<static_cast<unsigned>((keys + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pisa
