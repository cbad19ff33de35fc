// Per-head RMS norm of queries and keys with the rotation by position, forward and backward.
//
// Forward, per row x of d elements: y = x r w, r = rsqrt(mean x^2 + eps); the pairs of y's first
// `rot` elements turn by pos * inv_freq. Backward: g = the output's gradient turned back,
// dw += g x r, dx = r (g w) - x (r^3 / d) sum(g w x).
//
// Bound: memory (read and write once, 2 bytes an element each way). A row is held by d / 8 lanes,
// 16 bytes each, so the whole row stays in registers between the norm's reduction and the store;
// the half-split layout's partner elements come from another lane by shuffles of the raw bits.
// One warp takes one token and runs over its heads (Q's, then K's), several rows in flight, so the
// cosines and sines, and their products with the weights, are formed once per token. With few
// tokens (decode) the heads are split over warps instead: the work there is one round of latency.
//
// Angles: pos * inv_freq / (2 pi) is needed modulo 1, and a float product would lose the fraction
// of far positions (at position 10^6 by 0.03 turns). inv_freq / (2 pi) is held as a 64-bit binary
// fraction of a turn; its product with the position modulo 2^64 is exact integer arithmetic.
#include <algorithm>

#include "device.cuh"
#include "profile.h"
#include "window.h"

namespace pisa {

namespace {

constexpr int kWarps = 8;
constexpr int kInFlight = 4;     // rows of a lane group loaded before the first is used

struct RopeArgs {
  RopeDims s;
  const __nv_bfloat16* x[2];     // Q, K
  const __nv_bfloat16* dy[2];    // dQr, dKr (backward)
  __nv_bfloat16* y[2];           // outputs: Qr, Kr or dQ, dK
  const float* w[2];
  const float* inv_freq;
  const int32_t* pos;
  float* partial;                // backward: [blocks][2][d] sums of dw, or NULL
  int32_t* status;               // backward: the workspace's status word, cleared
  int32_t heads_per_warp;
  int64_t tokens;
};

// x / (2 pi) as a 64-bit fraction of a turn (modulo 1): x = m 2^e with a 24-bit m, times the
// first 64 binary digits of 1 / (2 pi).
__device__ __forceinline__ uint64_t turns64(float x) {
  const uint32_t bits = __float_as_uint(x);
  const int ex = (bits >> 23) & 255;
  const uint64_t m = ex ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const uint64_t inv2pi = 0x28BE60DB9391054Aull;
  const uint64_t lo = m * inv2pi, hi = __umul64hi(m, inv2pi);
  const int sh = 150 - (ex ? ex : 1);            // x = m 2^-sh
  uint64_t t;
  if (sh <= 0) t = sh > -64 ? lo << -sh : 0;
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

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(r[k] << 16);
    v[2 * k + 1] = __uint_as_float(r[k] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// Sum over the D / 8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// This lane's 8 elements of a row, with where they turn: IL (interleaved) pairs lie inside the
// lane; otherwise the partner elements are those of lane `partner`.
template <int D, bool IL>
struct Lane {
  int c, partner;
  bool turns, second;
  uint64_t inc[IL ? 4 : 8];

  __device__ __forceinline__ Lane(int lane, int rot, const float* inv_freq) {
    c = lane % (D / 8);
    turns = 8 * c < rot;
    second = !IL && 16 * c >= rot;
    partner = IL || !turns ? lane : second ? lane - rot / 16 : lane + rot / 16;
    const int f0 = IL ? 4 * c : 8 * c - (second ? rot / 2 : 0);
#pragma unroll
    for (int k = 0; k < (IL ? 4 : 8); ++k) inc[k] = turns ? turns64(inv_freq[f0 + k]) : 0;
  }
  // The partner's raw bits (zero where nothing turns, so that an infinity there stays itself).
  __device__ __forceinline__ uint4 other(const uint4& u) const {
    if (IL) return u;
    uint4 p;
    p.x = __shfl_sync(0xffffffffu, u.x, partner);
    p.y = __shfl_sync(0xffffffffu, u.y, partner);
    p.z = __shfl_sync(0xffffffffu, u.z, partner);
    p.w = __shfl_sync(0xffffffffu, u.w, partner);
    return turns ? p : make_uint4(0, 0, 0, 0);
  }
  // Per element: cos and the partner's factor (+-sin), times rot_scale; 1 and 0 where nothing turns.
  __device__ __forceinline__ void factors(int pos, float scale, bool back, float (&a)[8], float (&b)[8]) const {
#pragma unroll
    for (int k = 0; k < (IL ? 4 : 8); ++k) {
      float cs, sn;
      turn(inc[k], pos, scale, cs, sn);
      if (back) sn = -sn;
      if (!turns) { cs = 1.f; sn = 0.f; }
      if (IL) {
        a[2 * k] = a[2 * k + 1] = cs;
        b[2 * k] = -sn;
        b[2 * k + 1] = sn;
      } else {
        a[k] = cs;
        b[k] = second ? sn : -sn;
      }
    }
  }
};

template <bool IL>
__device__ __forceinline__ float partner_of(const float (&v)[8], const float (&p)[8], int e) {
  return IL ? v[e ^ 1] : p[e];
}

// The turned values: v a + partner b. (Interleaved elements that do not turn have b = 0, and their
// partner is left out so that an infinity there stays itself.)
template <bool IL>
__device__ __forceinline__ float turned(const float (&v)[8], const float (&p)[8], const float (&a)[8],
                                        const float (&b)[8], int e, bool turns) {
  if (IL) return turns ? v[e] * a[e] + v[e ^ 1] * b[e] : v[e] * a[e];
  return v[e] * a[e] + p[e] * b[e];
}

template <int D, bool IL, bool NORM>
__global__ void __launch_bounds__(32 * kWarps, 2) rope_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const RopeDims& s = a.s;
  const int lane = threadIdx.x & 31, g = lane / LPR;
  const Lane<D, IL> L(lane, s.rot, a.inv_freq);
  const int H = s.Hq + s.Hkv, hpw = a.heads_per_warp, chunks = (H + hpw - 1) / hpw;
  const int64_t work = a.tokens * chunks;
  for (int64_t wk = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); wk < work;
       wk += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t t = wk / chunks;
    const int h_beg = static_cast<int>(wk % chunks) * hpw, h_end = min(H, h_beg + hpw);
    const int pos = a.pos ? a.pos[t] : static_cast<int>(t % s.N);
    float ca[8], cb[8];
    L.factors(pos, s.rot_scale, false, ca, cb);
#pragma unroll
    for (int part = 0; part < 2; ++part) {                 // Q's heads, then K's
      const int Hx = part ? s.Hkv : s.Hq, off = part ? s.Hq : 0;
      const int lo = max(h_beg - off, 0), hi = min(h_end - off, Hx);
      if (lo >= hi) continue;
      float wa[8], wb[8];                                  // weight times factor, own and partner's
#pragma unroll
      for (int e = 0; e < 8; ++e) wa[e] = NORM && a.w[part] ? a.w[part][8 * L.c + e] : 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float wp = IL ? wa[e ^ 1] : __shfl_sync(0xffffffffu, wa[e], L.partner);
        wb[e] = cb[e] * wp;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) wa[e] *= ca[e];
      const __nv_bfloat16* x = a.x[part] + t * (part ? s.ks : s.qs) + 8 * L.c;
      __nv_bfloat16* y = a.y[part] + t * Hx * D + 8 * L.c;
      for (int h0 = lo; h0 < hi; h0 += RPW * kInFlight) {
        uint4 u[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
          const int h = h0 + k * RPW + g;
          u[k] = h < hi ? *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(h) * D) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
          const int h = h0 + k * RPW + g;
          if (h0 + k * RPW >= hi) break;                   // the same for the whole warp
          float v[8], p[8], o[8];
          unpack8(u[k], v);
          unpack8(L.other(u[k]), p);
          float r = 1.f;
          if (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
            r = rsqrtf(row_sum<D>(ss) * (1.f / D) + s.eps);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float z = turned<IL>(v, p, wa, wb, e, L.turns);
            o[e] = NORM ? z * r : z;
          }
          if (h < hi) *reinterpret_cast<uint4*>(y + static_cast<int64_t>(h) * D) = pack8(o);
        }
      }
    }
  }
}

template <int D, bool IL, bool NORM>
__global__ void __launch_bounds__(32 * kWarps, 2) rope_bwd_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  __shared__ float red[NORM ? kWarps : 1][2][D];
  const RopeDims& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / LPR;
  const Lane<D, IL> L(lane, s.rot, a.inv_freq);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.tokens;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int pos = a.pos ? a.pos[t] : static_cast<int>(t % s.N);
    float ca[8], cb[8];
    L.factors(pos, s.rot_scale, true, ca, cb);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int Hx = part ? s.Hkv : s.Hq;
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = NORM && a.w[part] ? a.w[part][8 * L.c + e] : 1.f;
      const __nv_bfloat16* x = a.x[part] + t * (part ? s.ks : s.qs) + 8 * L.c;
      const __nv_bfloat16* dy = a.dy[part] + t * Hx * D + 8 * L.c;
      __nv_bfloat16* y = a.y[part] + t * Hx * D + 8 * L.c;
      constexpr int F = kInFlight / 2;                     // two tensors are read
      for (int h0 = 0; h0 < Hx; h0 += RPW * F) {
        uint4 u[F], ux[F];
#pragma unroll
        for (int k = 0; k < F; ++k) {
          const int h = h0 + k * RPW + g;
          const bool ok = h < Hx;
          u[k] = ok ? *reinterpret_cast<const uint4*>(dy + static_cast<int64_t>(h) * D) : make_uint4(0, 0, 0, 0);
          ux[k] = NORM && ok ? *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(h) * D) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < F; ++k) {
          const int h = h0 + k * RPW + g;
          if (h0 + k * RPW >= Hx) break;
          float v[8], p[8], gr[8], xv[8];
          unpack8(u[k], v);
          unpack8(L.other(u[k]), p);
#pragma unroll
          for (int e = 0; e < 8; ++e) gr[e] = turned<IL>(v, p, ca, cb, e, L.turns);
          if (NORM) {
            unpack8(ux[k], xv);
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              ss += xv[e] * xv[e];
              dot += gr[e] * w[e] * xv[e];
            }
            const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + s.eps);
            const float m = row_sum<D>(dot) * (1.f / D) * r * r * r;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              dw[part][e] += gr[e] * xv[e] * r;
              gr[e] = r * gr[e] * w[e] - xv[e] * m;
            }
          }
          if (h < Hx) *reinterpret_cast<uint4*>(y + static_cast<int64_t>(h) * D) = pack8(gr);
        }
      }
    }
  }
  if (NORM && a.partial) {       // the block's sums: lane groups by shuffles, then warps in order
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = dw[part][e];
#pragma unroll
        for (int o = 16; o >= LPR; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane < LPR) red[warp][part][8 * L.c + e] = v;
      }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * D; k += 32 * kWarps) {
      float v = 0.f;
      for (int w = 0; w < kWarps; ++w) v += red[w][k / D][k % D];
      a.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + k] = v;
    }
  }
}

// dw[part][e] = sum over the blocks' partials, in a fixed order: 8 interleaved runs, then those.
template <int D>
__global__ void __launch_bounds__(8 * D) rope_dw_kernel(const float* partial, int blocks, float* dwq, float* dwk) {
  __shared__ float red[8][D];
  const int part = blockIdx.x, e = threadIdx.x % D, run = threadIdx.x / D;
  float v = 0.f;
  for (int k = run; k < blocks; k += 8) v += partial[(static_cast<int64_t>(k) * 2 + part) * D + e];
  red[run][e] = v;
  __syncthreads();
  float* out = part ? dwk : dwq;
  if (run == 0 && out) {
    for (int k = 1; k < 8; ++k) v += red[k][e];
    out[e] = v;
  }
}

constexpr int kBlocksPerSm = 2;

int bwd_blocks(const RopeDims& s) {
  const int64_t need = (static_cast<int64_t>(s.B) * s.N + kWarps - 1) / kWarps;
  return static_cast<int>(std::min<int64_t>(need, 152 * kBlocksPerSm));
}

template <template <int, bool, bool> class Launch, class... A>
int by_kind(const RopeDims& s, A... args) {
  if (s.d == 128) {
    if (s.interleaved) return s.norm ? Launch<128, true, true>::run(args...) : Launch<128, true, false>::run(args...);
    return s.norm ? Launch<128, false, true>::run(args...) : Launch<128, false, false>::run(args...);
  }
  if (s.interleaved) return s.norm ? Launch<64, true, true>::run(args...) : Launch<64, true, false>::run(args...);
  return s.norm ? Launch<64, false, true>::run(args...) : Launch<64, false, false>::run(args...);
}

template <int D, bool IL, bool NORM>
struct FwdLaunch {
  static int run(const RopeArgs& a, int blocks, cudaStream_t st) {
    ProfScope ps(st, "qk_norm_rope");
    rope_kernel<D, IL, NORM><<<blocks, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
  }
};

template <int D, bool IL, bool NORM>
struct BwdLaunch {
  static int run(const RopeArgs& a, int blocks, float* dwq, float* dwk, cudaStream_t st) {
    {
      ProfScope ps(st, "qk_norm_rope_bwd");
      rope_bwd_kernel<D, IL, NORM><<<blocks, 32 * kWarps, 0, st>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.partial) return e;
    ProfScope ps(st, "qk_norm_rope_dw");
    rope_dw_kernel<D><<<2, 8 * D, 0, st>>>(a.partial, blocks, dwq, dwk);
    return cudaGetLastError();
  }
};

RopeArgs make_args(const RopeDims& s, const void* Q, const void* K, const float* inv_freq, const float* wq,
                   const float* wk, const int32_t* pos) {
  RopeArgs a{};
  a.s = s;
  a.x[0] = static_cast<const __nv_bfloat16*>(Q);
  a.x[1] = static_cast<const __nv_bfloat16*>(K);
  a.w[0] = wq;
  a.w[1] = wk;
  a.inv_freq = inv_freq;
  a.pos = pos;
  a.tokens = static_cast<int64_t>(s.B) * s.N;
  return a;
}

}  // namespace

size_t rope_bwd_ws(const RopeDims& s) {
  return 256 + static_cast<size_t>(bwd_blocks(s)) * 2 * s.d * sizeof(float);
}

int launch_rope(const RopeDims& s, const void* Q, const void* K, const float* inv_freq, const float* wq,
                const float* wk, const int32_t* pos, void* Qr, void* Kr, void* stream) {
  RopeArgs a = make_args(s, Q, K, inv_freq, wq, wk, pos);
  a.y[0] = static_cast<__nv_bfloat16*>(Qr);
  a.y[1] = static_cast<__nv_bfloat16*>(Kr);
  const int H = s.Hq + s.Hkv, rpw = 256 / s.d;
  // all heads of a token to one warp where the tokens alone fill the GPU's warps; else a warp
  // takes one round of rows
  const int64_t slots = 152 * kBlocksPerSm * kWarps;
  a.heads_per_warp = a.tokens >= slots ? H : rpw;
  const int64_t work = a.tokens * ((H + a.heads_per_warp - 1) / a.heads_per_warp);
  const int blocks = static_cast<int>(std::min<int64_t>((work + kWarps - 1) / kWarps, 152 * kBlocksPerSm));
  return by_kind<FwdLaunch>(s, a, blocks, static_cast<cudaStream_t>(stream));
}

int launch_rope_bwd(const RopeDims& s, const void* Q, const void* K, const void* dQr, const void* dKr,
                    const float* inv_freq, const float* wq, const float* wk, const int32_t* pos, void* dQ, void* dK,
                    float* dwq, float* dwk, char* ws, void* stream) {
  RopeArgs a = make_args(s, Q, K, inv_freq, wq, wk, pos);
  a.dy[0] = static_cast<const __nv_bfloat16*>(dQr);
  a.dy[1] = static_cast<const __nv_bfloat16*>(dKr);
  a.y[0] = static_cast<__nv_bfloat16*>(dQ);
  a.y[1] = static_cast<__nv_bfloat16*>(dK);
  a.status = reinterpret_cast<int32_t*>(ws);
  a.partial = dwq || dwk ? reinterpret_cast<float*>(ws + 256) : nullptr;
  return by_kind<BwdLaunch>(s, a, bwd_blocks(s), dwq, dwk, static_cast<cudaStream_t>(stream));
}

}  // namespace pisa
