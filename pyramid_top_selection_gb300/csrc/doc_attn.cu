// Attention over packed documents, forward and backward: one warp per (row, head), or (key, KV head), a pair at a time.
#include <cmath>

#include "device.cuh"
#include "internal.h"
#include "paged.h"
#include "profile.h"

namespace pisa {

namespace {

using bf16 = __nv_bfloat16;

struct DocArgs {
  DocDims s;
  DocMask m;
  const bf16 *Q, *K, *V, *O, *dO;
  const float* lse_in;
  float* lse;
  bf16 *out, *dQ, *dK, *dV;
};

// The document of token t: its tokens [start, end), and one past its prefix; start = end where there is none.
struct Doc {
  int start, end, pre;
  __device__ __forceinline__ Doc(const DocArgs& a, int t) {
    int lo = 0, hi = a.s.n_docs + 1;             // starts below lo are <= t, those from hi on are > t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.m.starts[mid] <= t) lo = mid + 1; else hi = mid;
    }
    start = end = pre = 0;
    if (lo == 0 || lo > a.s.n_docs) return;
    start = max(0, a.m.starts[lo - 1]);
    end = min(a.s.T, a.m.starts[lo]);
    pre = a.m.prefix ? min(end, static_cast<int>(min(static_cast<int64_t>(start) + a.m.prefix[lo - 1], int64_t(1) << 30))) : start;
  }
};

template <int D>
struct Row {
  float v[D / 32];
  __device__ __forceinline__ Row(const bf16* p, int lane) {
    for (int k = 0; k < D / 32; ++k) v[k] = __bfloat162float(p[lane + 32 * k]);
  }
  __device__ __forceinline__ float dot(const Row& o) const {
    float x = 0.f;
    for (int k = 0; k < D / 32; ++k) x += v[k] * o.v[k];
    return warp_sum(x);
  }
};

// Score of a pair from its scaled product, and the factor that a gradient takes through the cap.
__device__ __forceinline__ float score(const DocArgs& a, float x, int h, int i, int j, float& back) {
  back = 1.f;
  if (a.s.cap > 0.f) {
    const float t = tanhf(x / a.s.cap);
    back = 1.f - t * t;
    x = a.s.cap * t;
  }
  return a.m.slopes ? x - a.m.slopes[h] * fabsf(static_cast<float>(i - j)) : x;
}

template <int D, bool BWD>
__global__ void doc_row_kernel(const DocArgs a) {
  const DocDims& s = a.s;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(s.T) * s.Hq) return;
  const int t = static_cast<int>(w / s.Hq), h = static_cast<int>(w % s.Hq), kv = h / s.G;
  const Doc d(a, t);
  const int end = t < d.end ? max(t + 1, d.pre) : d.start;
  const Row<D> q(a.Q + t * s.qs + h * D, lane);
  float o[D / 32] = {}, m = neg_inf(), l = 0.f, delta = 0.f, back;
  if (BWD) delta = Row<D>(a.dO + w * D, lane).dot(Row<D>(a.O + w * D, lane));
  for (int j = d.start; j < end; ++j) {
    const Row<D> k(a.K + j * s.ks + kv * D, lane), v(a.V + j * s.vs + kv * D, lane);
    const float z = score(a, q.dot(k) * s.scale, h, t, j, back);
    if (BWD) {
      const float p = expf(z - a.lse_in[static_cast<int64_t>(h) * s.T + t]);
      const float ds = p * (Row<D>(a.dO + w * D, lane).dot(v) - delta) * back * s.scale;
      for (int k2 = 0; k2 < D / 32; ++k2) o[k2] += ds * k.v[k2];
    } else {
      const float mn = fmaxf(m, z), f = mn == neg_inf() ? 1.f : expf(m - mn), e = mn == neg_inf() ? 0.f : expf(z - mn);
      m = mn;
      l = l * f + e;
      for (int k2 = 0; k2 < D / 32; ++k2) o[k2] = o[k2] * f + e * v.v[k2];
    }
  }
  bf16* out = (BWD ? a.dQ : a.out) + w * D;
  for (int k = 0; k < D / 32; ++k) out[lane + 32 * k] = __float2bfloat16_rn(BWD ? o[k] : l == 0.f ? 0.f : o[k] / l);
  if (!BWD && lane == 0) a.lse[static_cast<int64_t>(h) * s.T + t] = l == 0.f ? neg_inf() : m + logf(l);
}

template <int D>
__global__ void doc_key_kernel(const DocArgs a) {
  const DocDims& s = a.s;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(s.T) * s.Hkv) return;
  const int j = static_cast<int>(w / s.Hkv), kv = static_cast<int>(w % s.Hkv);
  const Doc d(a, j);
  const bool in = j < d.end;
  const Row<D> k(a.K + j * s.ks + kv * D, lane), v(a.V + j * s.vs + kv * D, lane);
  float dk[D / 32] = {}, dv[D / 32] = {}, back;
  for (int i = in ? (j < d.pre ? d.start : j) : 0; i < (in ? d.end : 0); ++i)
    for (int h = kv * s.G; h < (kv + 1) * s.G; ++h) {
      const int64_t r = (static_cast<int64_t>(i) * s.Hq + h) * D;
      const Row<D> q(a.Q + i * s.qs + h * D, lane), g(a.dO + r, lane);
      const float p = expf(score(a, q.dot(k) * s.scale, h, i, j, back) - a.lse_in[static_cast<int64_t>(h) * s.T + i]);
      const float ds = p * (g.dot(v) - g.dot(Row<D>(a.O + r, lane))) * back * s.scale;
      for (int e = 0; e < D / 32; ++e) {
        dk[e] += ds * q.v[e];
        dv[e] += p * g.v[e];
      }
    }
  for (int e = 0; e < D / 32; ++e) {
    a.dK[w * D + lane + 32 * e] = __float2bfloat16_rn(dk[e]);
    a.dV[w * D + lane + 32 * e] = __float2bfloat16_rn(dv[e]);
  }
}

template <int D>
int bwd(const DocArgs& a, cudaStream_t st) {
  {
    ProfScope ps(st, "doc_dq");
    doc_row_kernel<D, true><<<static_cast<unsigned>((static_cast<int64_t>(a.s.T) * a.s.Hq + 3) / 4), 128, 0, st>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ProfScope ps(st, "doc_dkv");
  doc_key_kernel<D><<<static_cast<unsigned>((static_cast<int64_t>(a.s.T) * a.s.Hkv + 3) / 4), 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t doc_fwd_ws(const DocDims&) { return 256; }
size_t doc_bwd_ws(const DocDims&) { return 256; }

int launch_doc_fwd(const DocDims& s, const void* Q, const void* K, const void* V, const DocMask& m, void* O, float* lse,
                   char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DocArgs a{};
  a.s = s;
  a.m = m;
  a.Q = static_cast<const bf16*>(Q);
  a.K = static_cast<const bf16*>(K);
  a.V = static_cast<const bf16*>(V);
  a.out = static_cast<bf16*>(O);
  a.lse = lse;
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(s.T) * s.Hq + 3) / 4);
  ProfScope ps(st, "doc_fwd");
  if (s.d == 128) doc_row_kernel<128, false><<<blocks, 128, 0, st>>>(a);
  else doc_row_kernel<64, false><<<blocks, 128, 0, st>>>(a);
  return cudaGetLastError();
}

int launch_doc_bwd(const DocDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                   const void* dO, const DocMask& m, void* dQ, void* dK, void* dV, char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DocArgs a{};
  a.s = s;
  a.m = m;
  a.Q = static_cast<const bf16*>(Q);
  a.K = static_cast<const bf16*>(K);
  a.V = static_cast<const bf16*>(V);
  a.O = static_cast<const bf16*>(O);
  a.dO = static_cast<const bf16*>(dO);
  a.lse_in = lse;
  a.dQ = static_cast<bf16*>(dQ);
  a.dK = static_cast<bf16*>(dK);
  a.dV = static_cast<bf16*>(dV);
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return e;
  return s.d == 128 ? bwd<128>(a, st) : bwd<64>(a, st);
}

}  // namespace pisa
