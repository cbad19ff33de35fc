// What turns rows of queries and keys: angles in fixed point, and a row's elements as a lane holds them (the query/key
// norm with rotation, and the append to a paged cache).
#pragma once

#include "device.cuh"
#include "window_tc.cuh"

namespace pisa {
namespace rope {

using win::mul2;

// x / (2 pi) as a 64-bit fraction of a turn (modulo 1), for any finite x, to within 2^-63: x = m 2^-sh with a
// 24-bit m, times 128 of the first 256 binary digits of 1 / (2 pi). Where x is a multiple of 2^up, the first `up`
// digits make whole turns and are passed over. (The digits are immediates: read from constant memory they
// delayed the kernel's start by 1 us.)
__device__ __forceinline__ uint64_t turns64(float x) {
  const uint32_t bits = __float_as_uint(x);
  const int ex = (bits >> 23) & 255;
  const uint64_t m = ex ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int sh = 150 - (ex ? ex : 1), up = max(0, -sh);
  const bool far = up >= 64;
  const uint64_t d0 = far ? 0x7F09D5F47D4D3770ull : 0x28BE60DB9391054Aull, d1 = far ? 0x36D8A5664F10E410ull : 0x7F09D5F47D4D3770ull,
                 d2 = far ? 0x7F9458EAF7AEF158ull : 0x36D8A5664F10E410ull;
  auto digits = [&](uint64_t a, uint64_t b) { return up & 63 ? a << (up & 63) | b >> (64 - (up & 63)) : a; };
  const uint64_t first = digits(d0, d1), carry = __umul64hi(m, digits(d1, d2)), lo = m * first + carry,
                 hi = __umul64hi(m, first) + (lo < carry);
  uint64_t t;
  if (sh <= 0) t = lo;
  else if (sh < 64) t = (hi << (64 - sh)) | (lo >> sh);
  else t = sh < 128 ? hi >> (sh - 64) : 0;
  return bits >> 31 ? 0 - t : t;
}

// Cosine and sine of pos times the fraction `inc` of a turn, times m. The angle is reduced to
// [-pi, pi], where the fast functions' absolute error is below 2^-21: far under the bf16 outputs.
__device__ __forceinline__ void turn(uint64_t inc, int pos, float m, float& c, float& s) {
  const uint64_t ph = inc * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const float a = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 1.46291807926715968e-9f;   // 2 pi / 2^32
  __sincosf(a, &s, &c);
  c *= m;
  s *= m;
}

// Sum over the D / 8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's 8 elements of a row: two runs of four, `at` elements [0] and [1] from the row's start, whose
// k-th elements are a pair (first, second). Half-split: the runs lie rot / 2 apart. Interleaved
// (IL), and elements that do not turn: eight in a row (interleaved, the pairs are its even and odd ones).
// The warp forms a token's rot / 2 cosines and sines once, each lane two of them at most, in its
// table in shared memory.
template <int D, bool IL>
struct Lane {
  int at[2], f0, half;
  bool turns;
  uint64_t inc[D / 64];
  float2* tab;

  __device__ __forceinline__ Lane(int lane, int rot, const float* inv_freq, float2* table) {
    const int c = lane % (D / 8);
    half = rot / 2;
    turns = 8 * c < rot;
    at[0] = turns && !IL ? 4 * c : 8 * c;
    at[1] = turns && !IL ? half + 4 * c : 8 * c + 4;
    f0 = turns ? 4 * c : 0;
    tab = table;
#pragma unroll
    for (int k = 0; k < D / 64; ++k) inc[k] = lane + 32 * k < half ? turns64(inv_freq[lane + 32 * k]) : 0;
  }
  // Element k's place in the row (k < 4: first of pair k, else second of pair k - 4).
  __device__ __forceinline__ int element(int k) const { return IL ? at[0] + 2 * (k & 3) + (k >> 2) : at[k >> 2] + (k & 3); }
  // The table of one position, times rot_scale.
  __device__ __forceinline__ void form(int lane, int pos, float scale) const {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      if (lane + 32 * k < half) {
        float cs, sn;
        turn(inc[k], pos, scale, cs, sn);
        tab[lane + 32 * k] = make_float2(cs, sn);
      }
    __syncwarp();
  }
  // Cosines and sines of the lane's four pairs; 1 and 0 where nothing turns.
  __device__ __forceinline__ void factors(float (&c)[4], float (&s)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const float4 t = *reinterpret_cast<const float4*>(tab + f0 + k);
      c[k] = turns ? t.x : 1.f;
      s[k] = turns ? t.y : 0.f;
      c[k + 1] = turns ? t.z : 1.f;
      s[k + 1] = turns ? t.w : 0.f;
    }
  }
  // The lane's pairs of a row, and back: v[0], v[1] the firsts (two pairs each), v[2], v[3] the seconds.
  __device__ __forceinline__ void load(const unsigned char* row, uint64_t (&v)[4]) const {
    const uint2 a = *reinterpret_cast<const uint2*>(row + 2 * at[0]), b = *reinterpret_cast<const uint2*>(row + 2 * at[1]);
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
    float lo[4], hi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo[k] = __uint_as_float(w[k] << 16);
      hi[k] = __uint_as_float(w[k] & 0xffff0000u);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      v[k] = IL ? tc::pack2(lo[2 * k], lo[2 * k + 1]) : tc::pack2(lo[k], hi[k]);
      v[2 + k] = IL ? tc::pack2(hi[2 * k], hi[2 * k + 1]) : tc::pack2(lo[2 + k], hi[2 + k]);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, const uint64_t (&v)[4]) const {
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) tc::unpack2(v[k], x[2 * k], x[2 * k + 1]);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = IL ? pack_bf16(x[k], x[4 + k]) : pack_bf16(x[2 * k], x[2 * k + 1]);
    *reinterpret_cast<uint2*>(row + at[0]) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + at[1]) = make_uint2(w[2], w[3]);
  }
};

}  // namespace rope
}  // namespace pisa
