// Attention of the last tokens of every sequence over a paged cache in 16 or 4 bits: one warp per (sequence, query, head),
// a key at a time.
#include <cmath>

#include "internal.h"
#include "paged.cuh"
#include "profile.h"
#include "window_tc.cuh"

namespace pisa {

namespace {

using bf16 = __nv_bfloat16;

struct PagedArgs {
  PagedDims s;
  PagedCache c;
  const int32_t *table, *len;
  const bf16* q;
  const float* slopes;
  bf16* o;
  float* lse;
  int32_t* status;
};

template <int D>
__device__ __forceinline__ float element(const PagedDims& s, const unsigned char* p, const unsigned char* sc, int64_t row, int e) {
  if (s.bits == 16) return __bfloat162float(reinterpret_cast<const bf16*>(p)[row * D + e]);
  uint32_t h[4];
  paged::from_e2m1x8(p[row * (D / 2) + e / 2], h);
  const __half2 v = *reinterpret_cast<__half2*>(&h[0]);
  return __half2float(e & 1 ? __high2half(v) : __low2half(v)) * __low2float(paged::from_e4m3x2(sc[row * (D / 16) + e / 16]));
}

template <int D>
__global__ void paged_attn_kernel(const PagedArgs a) {
  const PagedDims& s = a.s;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(s.B) * s.nq * s.Hq) return;
  const int h = static_cast<int>(w % s.Hq), i = static_cast<int>(w / s.Hq % s.nq), b = static_cast<int>(w / s.Hq / s.nq), kv = h / s.G;
  const int most = s.max_pages << s.log_page, n0 = a.len[b], n = max(0, min(n0, most)), p = n - s.nq + i;
  if (n != n0 && lane == 0) atomicOr(a.status, PISA_STATUS_POS_RANGE);
  float q[D / 32], o[D / 32] = {}, m = neg_inf(), l = 0.f;
  for (int k = 0; k < D / 32; ++k) q[k] = __bfloat162float(a.q[w * D + lane + 32 * k]);
  const float ka = a.c.k_amp ? a.c.k_amp[kv] : 1.f, va = a.c.v_amp ? a.c.v_amp[kv] : 1.f, slope = a.slopes ? a.slopes[h] : 0.f;
  for (int j = 0; j <= p; ++j) {
    const int page = a.table[static_cast<int64_t>(b) * s.max_pages + (j >> s.log_page)];
    if (page < 0 || page >= s.n_pages) {
      if (lane == 0) atomicOr(a.status, PISA_STATUS_POS_RANGE);
      continue;
    }
    const int64_t row = (static_cast<int64_t>(page) * s.Hkv + kv) * s.page + (j & (s.page - 1));
    float x = 0.f;
    for (int k = 0; k < D / 32; ++k) x += q[k] * element<D>(s, a.c.k, a.c.ks, row, lane + 32 * k);
    x = warp_sum(x) * s.scale * ka;
    if (s.cap > 0.f) x = s.cap * tanhf(x / s.cap);
    x -= slope * static_cast<float>(p - j);
    const float mn = fmaxf(m, x), f = mn == neg_inf() ? 1.f : expf(m - mn), e = mn == neg_inf() ? 0.f : expf(x - mn);
    m = mn;
    l = l * f + e;
    for (int k = 0; k < D / 32; ++k) o[k] = o[k] * f + e * element<D>(s, a.c.v, a.c.vs, row, lane + 32 * k);
  }
  for (int k = 0; k < D / 32; ++k) a.o[w * D + lane + 32 * k] = __float2bfloat16_rn(l == 0.f ? 0.f : o[k] * va / l);
  if (lane == 0 && a.lse) a.lse[w] = l == 0.f ? neg_inf() : m + logf(l);
}

}  // namespace

size_t paged_attn_ws(const PagedDims&) { return 256; }

int launch_paged_attn(const PagedDims& s, const PagedCache& c, const int32_t* table, const int32_t* len, const void* q,
                      const float* slopes, void* o, float* lse, char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const PagedArgs a{s, c, table, len, static_cast<const bf16*>(q), slopes, static_cast<bf16*>(o), lse, reinterpret_cast<int32_t*>(ws)};
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(s.B) * s.nq * s.Hq + 3) / 4);
  ProfScope ps(st, "paged_attn");
  if (s.d == 128) paged_attn_kernel<128><<<blocks, 128, 0, st>>>(a);
  else paged_attn_kernel<64><<<blocks, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pisa
