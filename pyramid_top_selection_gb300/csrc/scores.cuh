// Scores of the documents' attention and of the paged cache's: cap tanh(x / cap), less a slope times the distance.
#pragma once

#include "tc.cuh"

namespace pisa {

constexpr float kScoreLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh within 2^-22 of 1, and within 2^-23 of itself for |x| <= 1/4: its series there, elsewhere
// 1 - 2 / (1 + e^(2 |x|)), whose difference of near numbers would cost small x their digits.
__device__ __forceinline__ float tanh_of(float x) {
  const float a = fabsf(x), y = x * x;
  const float small = x + x * y * fmaf(y, fmaf(y, fmaf(y, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f);
  const float big = 1.f - 2.f * rcp_approx(1.f + tc::ex2(a * (2.f * kScoreLog2e)));
  return a <= 0.25f ? small : copysignf(big, x);
}

}  // namespace pisa
