// Rows of the documents' attention taken pair by pair, for values that are not finite.
//
// The tensor cores' products take a whole tile: what a row does not see has a weight of 0 there, and 0 times an infinity or a
// NaN is NaN. So one document's bad token would reach its neighbours', and a row the ones behind it, wherever they share a tile.
// The kernels therefore look at what they put out (a multiply-add for two values); where that is not finite and something that
// the row does not see is not finite either, a warp forms the row again from the pairs that it does see, before the kernel
// ends. Nothing of this runs where values are finite; its code and the look at the outputs cost no more than 1.5 % (six prompts capped
// 677 -> 680 us, 60 documents capped 286 -> 290, not capped 187 -> 190). With one infinity a forward of six prompts takes 23 ms instead
// of 0.7, and a training pass of 60 documents of up to 2048 tokens 3.7 instead of 0.8; with a channel of infinities 124 and 63.
#pragma once

#include "device.cuh"
#include "masks.cuh"

namespace pisa {
namespace win {

// Whether all values that were added are finite (their sum times 0 is 0): four sums, which do not wait for one another.
struct Watch {
  uint64_t sum[4];
  __device__ __forceinline__ Watch() : sum{0, 0, 0, 0} {}
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 2) sum[c >> 1 & 3] = tc::fma2(tc::pack2(x[c], x[c + 1]), 0ull, sum[c >> 1 & 3]);
  }
  __device__ __forceinline__ bool bad() const {
    float a, b;
    tc::unpack2(tc::add2(tc::add2(sum[0], sum[1]), tc::add2(sum[2], sum[3])), a, b);
    return !(a + b == 0.f);
  }
};

// What this warp's bulk stores wrote, and it has waited for, can be read.
__device__ __forceinline__ void fence_async_global() {
  __syncwarp();
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

// Whether one of eight (two) bf16 values is not finite.
__device__ __forceinline__ bool not_finite(uint32_t v) {
  v &= 0x7fff7fffu;
  return (v & 0xffffu) >= 0x7f80u || (v >> 16) >= 0x7f80u;
}
__device__ __forceinline__ bool not_finite(uint4 v) {
  const uint32_t m = 0x7fff7fffu;
  return not_finite(__vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m)));
}
// Of a row of D values (one lane), and of rows [from, to), `stride` elements apart (whole warp).
template <int D>
__device__ __forceinline__ bool row_not_finite(const __nv_bfloat16* row) {
  bool bad = false;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) bad |= not_finite(*reinterpret_cast<const uint4*>(row + 8 * c));
  return bad;
}
template <int D>
__device__ __forceinline__ bool rows_not_finite(const __nv_bfloat16* rows, int64_t stride, int from, int to) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int r0 = from; r0 < to; r0 += RPW) {
    const int r = r0 + lane / LPR;
    if (__any_sync(0xffffffffu, r < to && not_finite(ldg_u4(rows + r * stride + lane % LPR * 8)))) return true;
  }
  return false;
}

// The product of two rows (one lane).
template <int D>
__device__ __forceinline__ float row_product(const __nv_bfloat16* a, const __nv_bfloat16* b) {
  float s = 0.f;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = ldg_u4(a + 8 * c), y = ldg_u4(b + 8 * c);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(xw[e] << 16), __uint_as_float(yw[e] << 16), s);
      s = fmaf(__uint_as_float(xw[e] & 0xffff0000u), __uint_as_float(yw[e] & 0xffff0000u), s);
    }
  }
  return s;
}

// The warp's sum of weights times rows: lane l holds values D / 32 l ...
template <int D>
struct RowSum {
  static constexpr int E = D / 32;
  float v[E];
  __device__ __forceinline__ RowSum() {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
  }
  // lane k's weight times row k (stride elements apart), k < n
  __device__ __forceinline__ void add(float weight, const __nv_bfloat16* rows, int64_t stride, int n) {
    const __nv_bfloat16* at = rows + E * (threadIdx.x & 31);
#pragma unroll 4
    for (int k = 0; k < n; ++k, at += stride) {
      const float w = __shfl_sync(0xffffffffu, weight, k);
      uint32_t u[E / 2];
      if constexpr (E == 4) {
        const uint2 x = ldg_u2(at);
        u[0] = x.x;
        u[E / 2 - 1] = x.y;
      } else {
        u[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
      }
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        v[2 * e] = fmaf(w, __uint_as_float(u[e] << 16), v[2 * e]);
        v[2 * e + 1] = fmaf(w, __uint_as_float(u[e] & 0xffff0000u), v[2 * e + 1]);
      }
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, float f) const {
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(row + E * (threadIdx.x & 31) + e) = pack_bf16(f * v[e], f * v[e + 1]);
  }
  __device__ __forceinline__ void store(float* row, float f) const {
#pragma unroll
    for (int e = 0; e < E; ++e) row[E * (threadIdx.x & 31) + e] = f * v[e];
  }
  // Whether the warp's row holds what is not finite.
  static __device__ __forceinline__ bool bad(const __nv_bfloat16* row) {
    bool b = false;
#pragma unroll
    for (int e = 0; e < E; e += 2) b |= not_finite(*reinterpret_cast<const uint32_t*>(row + E * (threadIdx.x & 31) + e));
    return __any_sync(0xffffffffu, b);
  }
  static __device__ __forceinline__ bool bad(const float* row) {
    bool b = false;
#pragma unroll
    for (int e = 0; e < E; ++e) b |= !isfinite(row[E * (threadIdx.x & 31) + e]);
    return __any_sync(0xffffffffu, b);
  }
};

// A pair's score in powers of two, as Scores and Distance have it for tiles; back: what a gradient takes through the cap.
template <int MASK>
__device__ __forceinline__ float pair_score(float x, float scale, float cap, float slope2, int distance, float& back) {
  float y = x * (scale * kScoreLog2e);
  back = 1.f;
  if (MASK & kCap) {
    const float t = tanh_of(x * (scale / cap));
    y = cap * kScoreLog2e * t;
    back = 1.f - t * t;
  }
  if (MASK & kBias) y -= slope2 * static_cast<float>(abs(distance));
  return y;
}

}  // namespace win
}  // namespace pisa
