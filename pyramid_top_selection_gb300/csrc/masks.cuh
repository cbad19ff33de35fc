// What the rows of the tensor-core attention see, and what becomes of their scores: a window with sinks, or the document
// that a row belongs to, with scores as they are or capped and biased by distance. The forward and backward kernels
// (window_fwd.cuh, window_bwd.cuh) take one of these as a template argument.
#pragma once

#include "scores.cuh"
#include "window_tc.cuh"

namespace pisa {
namespace win {

constexpr int kWindow = 0, kDocs = 1, kScored = 2;

// Documents on the device, as the prologue (doc_attn.cu) lays them out.
struct DocRows {
  const int4* bounds;      // [T + 1]: of a token: its document's tokens [x, y), one past its prefix z (x = y = z past the token: none).
                           // [T]: x the first document's first token, y one past the last one's
  const int32_t* order;    // token tiles, those with the most keys first
  const float* slopes;     // per query head, or NULL
  float cap;               // 0: none
};

// The keys [lo, hi] that token t sees (hi < lo: none).
struct DocSpan {
  int lo, hi;
  __device__ __forceinline__ DocSpan() : lo(0), hi(-1) {}
  __device__ __forceinline__ DocSpan(const DocRows& d, int t) {
    const int4 b = d.bounds[t];
    lo = b.x;
    hi = t < b.y ? max(t, b.z - 1) : -1;
  }
};

// The keys [lo, hi] that some token of [t0, t1) sees: spans neither begin nor end before an earlier token's.
struct DocRange {
  int lo, hi;
  __device__ __forceinline__ DocRange(const DocRows& d, int t0, int t1) : lo(0), hi(-1) {
    if (t0 >= t1) return;
    const int4 a = d.bounds[t0], z = d.bounds[t1 - 1];
    lo = a.x;
    hi = t1 - 1 < z.y ? max(t1 - 1, z.z - 1) : z.y - 1;
  }
};

// The tokens [first, end) that see key j.
struct DocSeen {
  int first, end;
  __device__ __forceinline__ DocSeen(const DocRows& d, int j, int T) : first(0), end(0) {
    if (j >= T) return;
    const int4 b = d.bounds[j];
    if (j >= b.y || j < b.x) return;
    first = j < b.z ? b.x : j;
    end = b.y;
  }
};

// Scores in powers of two of a thread's products x (a row's against columns, or a key's against rows).
//   y = cap tanh(k x), k = scale / cap: within |k x| <= 1 by a polynomial of (k x)^2 on the FMA units (minimax on [0, 1]:
//   tanh within 2.5e-7), as a warp that has no larger product takes it; else by tanh_of, three special-function operations.
// The polynomial's coefficients are taken times k^2i and scale log2 e, so that y = x p(x^2).
struct Scores {
  float c1, k, cap2;       // scale log2 e, scale / cap, cap log2 e
  float p[6];
  __device__ __forceinline__ Scores(float scale, float cap) : c1(scale * kScoreLog2e), k(0.f), cap2(cap * kScoreLog2e) {
    if (cap > 0.f) {
      k = scale / cap;
      const float k2 = k * k;
      const float c[6] = {0.999996841f, -0.333240032f, 0.132535249f, -0.0509728603f, 0.016114179f, -0.00283946446f};
      float f = c1;
#pragma unroll
      for (int i = 0; i < 6; ++i, f *= k2) p[i] = c[i] * f;
    }
  }
  // Whether a warp's products are within the polynomial's range.
  template <int N>
  __device__ __forceinline__ bool near(const float (&x)[N]) const {
    float top[4] = {fabsf(x[0]), fabsf(x[1]), fabsf(x[2]), fabsf(x[3])};
#pragma unroll
    for (int c = 4; c < N; c += 4)
#pragma unroll
      for (int q = 0; q < 4; ++q) top[q] = fmaxf(top[q], fabsf(x[c + q]));
    return __all_sync(0xffffffffu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * k <= 1.f);   // (NaN: not)
  }
  // Two scores before the distance's share.
  template <bool NEAR>
  __device__ __forceinline__ void capped(float& a, float& b) const {
    if (NEAR) {
      const uint64_t x = tc::pack2(a, b), y = mul2(x, x);
      uint64_t r = tc::pack2(p[5], p[5]);
#pragma unroll
      for (int i = 4; i >= 0; --i) r = tc::fma2(r, y, tc::pack2(p[i], p[i]));
      tc::unpack2(mul2(x, r), a, b);
    } else {
      a = cap2 * tanh_of(a * k);
      b = cap2 * tanh_of(b * k);
    }
  }
  // All of a thread's scores before the distance's share.
  template <int N>
  __device__ __forceinline__ void cap_all(float (&x)[N]) const {
    if (cap2 == 0.f) {
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] *= c1;
    } else if (near(x)) {
#pragma unroll
      for (int c = 0; c < N; c += 2) capped<true>(x[c], x[c + 1]);
    } else {
#pragma unroll
      for (int c = 0; c < N; c += 2) capped<false>(x[c], x[c + 1]);
    }
  }
  // What a gradient takes through the cap, from a capped score: 1 - tanh^2.
  __device__ __forceinline__ float back(float y, float icap2) const {
    const float t = y * icap2;
    return fmaf(-t, t, 1.f);
  }
};

}  // namespace win
}  // namespace pisa
