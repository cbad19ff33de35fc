// Per-head RMS norm of queries and keys with the rotation by position, forward and backward.
//
// Forward, per row x of d elements: y = x r w, r = rsqrt(mean x^2 + eps); the pairs of y's first
// `rot` elements turn by pos * inv_freq. Backward: g = the output's gradient turned back,
// dw += g x r, dx = r (g w) - x (r^3 / d) sum(g w x).
//
// Bound: memory (read and write once, 2 bytes an element each way); the 64K prefill's 16 + 2 heads of
// 128 take 98 us, 6.2 TB/s, the 16K training batch's 16 + 4 heads 111 us forward and 169 us backward.
// One warp takes one token and runs over its heads, Q's then K's, so that the cosines and sines, and
// their products with the weights, are formed once per token. A row is held by d / 8 lanes, each with
// both elements of its four pairs (in the half-split layout two runs of 8 bytes that lie rot / 2 apart),
// so that a pair turns within a lane; as 16 bytes a lane in a row, with the partners fetched by shuffles,
// the same 64K took 138 us. Rows come by cp.async into a ring of each warp's, two steps of four rounds
// (2 KB each) ahead of the arithmetic: with loads into registers instead, the warps waited for memory
// (the registers hold too few rows ahead). With few tokens (decode) the heads are split over warps
// instead: the work there is one round of latency.
//
// Angles: pos * inv_freq / (2 pi) is needed modulo 1, and a float product would lose the fraction
// of far positions (at position 10^6 by 0.03 turns). inv_freq / (2 pi) is held as a 64-bit binary
// fraction of a turn, of which its product with the position keeps 32 bits exactly (2^-63 of a turn off times
// 2^31: within 2^-31 of a turn for every position and frequency, cut to 32 bits included).
#include <algorithm>

#include "device.cuh"
#include "internal.h"
#include "profile.h"
#include "window_tc.cuh"

namespace pisa {

namespace {

constexpr int kWarps = 8;
constexpr int kFwdBlocks = 3, kBwdBlocks = 2;     // blocks an SM holds, by registers
constexpr int kRound = 4;        // row rounds (512 bytes a warp) of a step
constexpr int kAhead = 3;        // steps in a warp's ring: two in flight, one in use

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

using win::mul2;

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

// A warp's rows in order: its tokens' heads, Q's then K's, as steps of up to ROWS rows (a step does not
// cross from Q to K). Rows are loaded a step or more before their arithmetic, by cp.async into a ring of
// the warp's in shared memory.
struct Cursor {
  int64_t wk;        // unit of work: token * chunks + chunk of heads
  int part, h, end;  // Q or K, the step's first head, one past the part's last
};

template <int ROWS>
struct Walk {
  const RopeArgs& a;
  int hpw, chunks;
  int64_t work, step;
  __device__ __forceinline__ Walk(const RopeArgs& args)
      : a(args), hpw(args.heads_per_warp), chunks((args.s.Hq + args.s.Hkv + args.heads_per_warp - 1) / args.heads_per_warp),
        work(args.tokens * chunks), step(static_cast<int64_t>(gridDim.x) * kWarps) {}
  __device__ __forceinline__ int64_t token(const Cursor& c) const { return chunks == 1 ? c.wk : c.wk / chunks; }
  __device__ __forceinline__ int first_head(const Cursor& c) const { return chunks == 1 ? 0 : static_cast<int>(c.wk % chunks) * hpw; }
  __device__ __forceinline__ void open(Cursor& c) const {          // the first step of unit c.wk
    const int beg = first_head(c);
    c.part = beg >= a.s.Hq;
    c.h = beg - (c.part ? a.s.Hq : 0);
    c.end = c.part ? min(a.s.Hkv, c.h + hpw) : min(a.s.Hq, beg + hpw);
  }
  __device__ __forceinline__ void next(Cursor& c) const {
    c.h += ROWS;
    if (c.h < c.end) return;
    if (c.part == 0) {
      const int beg = first_head(c);
      if (beg + hpw > a.s.Hq) {
        c.part = 1;
        c.h = 0;
        c.end = min(a.s.Hkv, beg + hpw - a.s.Hq);
        return;
      }
    }
    c.wk += step;
    open(c);
  }
};

// Copies the step's rows (those below c.end) of a tensor into `dst`, D elements each.
template <int D>
__device__ __forceinline__ void fetch_rows(uint32_t dst, const __nv_bfloat16* x, const Cursor& c, int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int g = lane / LPR, e = 8 * (lane % LPR);
#pragma unroll
  for (int k = 0; k < kRound; ++k) {
    const int r = k * RPW + g;
    if (c.h + r < c.end) tc::cp_async16(dst + (r * D + e) * 2, x + static_cast<int64_t>(c.h + r) * D + e, true);
  }
}

template <int D, bool IL, bool NORM>
__global__ void __launch_bounds__(32 * kWarps, kFwdBlocks) rope_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kRound * 512;
  extern __shared__ __align__(16) unsigned char ring_all[];
  __shared__ __align__(16) float2 table[kWarps][D / 2];
  const RopeDims& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / LPR;
  unsigned char* ring = ring_all + warp * kAhead * STEP;
  const Lane<D, IL> L(lane, s.rot, a.inv_freq, table[warp]);
  const Walk<RPW * kRound> walk(a);
  Cursor c{static_cast<int64_t>(blockIdx.x) * kWarps + warp, 0, 0, 0};
  walk.open(c);
  Cursor f = c;
  auto fetch = [&](int slot) {
    if (f.wk < walk.work) {
      fetch_rows<D>(tc::su32(ring + slot * STEP), a.x[f.part] + walk.token(f) * (f.part ? s.ks : s.qs), f, lane);
      walk.next(f);
    }
    tc::cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) fetch(k);
  int64_t now = -1;                                        // the unit and part that the factors are for
  int now_part = 0;
  uint64_t aa[2], ab[2], ba[2], bb[2];                     // first = aa first + ab second, second = ba first + bb second
  for (int slot = 0; c.wk < walk.work; slot = slot + 1 == kAhead ? 0 : slot + 1) {
    const int64_t t = walk.token(c);
    if (c.wk != now || c.part != now_part) {
      if (c.wk != now) L.form(lane, a.pos ? a.pos[t] : static_cast<int>(t % s.N), s.rot_scale);
      now = c.wk;
      now_part = c.part;
      float cs[4], sn[4], w[8];
      L.factors(cs, sn);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = NORM && a.w[c.part] ? a.w[c.part][L.element(k)] : 1.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        aa[k] = tc::pack2(w[2 * k] * cs[2 * k], w[2 * k + 1] * cs[2 * k + 1]);
        ab[k] = tc::pack2(-w[4 + 2 * k] * sn[2 * k], -w[5 + 2 * k] * sn[2 * k + 1]);
        ba[k] = tc::pack2(w[2 * k] * sn[2 * k], w[2 * k + 1] * sn[2 * k + 1]);
        bb[k] = tc::pack2(w[4 + 2 * k] * cs[2 * k], w[5 + 2 * k] * cs[2 * k + 1]);
      }
    }
    tc::cp_async_wait<kAhead - 2>();
    __syncwarp();                                          // also: every lane has read the slot fetched next
    fetch(slot == 0 ? kAhead - 1 : slot - 1);
    const unsigned char* rows = ring + slot * STEP;
    __nv_bfloat16* y = a.y[c.part] + (t * (c.part ? s.Hkv : s.Hq) + c.h + g) * D;
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
      if (c.h + k * RPW >= c.end) break;                   // the same for the whole warp
      uint64_t v[4], o[4];
      L.load(rows + (k * RPW + g) * D * 2, v);
      uint64_t r2 = 0;
      if (NORM) {
        const uint64_t q = tc::fma2(v[3], v[3], tc::fma2(v[2], v[2], tc::fma2(v[1], v[1], mul2(v[0], v[0]))));
        float q0, q1;
        tc::unpack2(q, q0, q1);
        const float r = rsqrtf(row_sum<D>(q0 + q1) * (1.f / D) + s.eps);
        r2 = tc::pack2(r, r);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // what does not turn does not meet its partner, so that an infinity there stays itself
        o[e] = L.turns ? tc::fma2(v[2 + e], ab[e], mul2(v[e], aa[e])) : mul2(v[e], aa[e]);
        o[2 + e] = L.turns ? tc::fma2(v[e], ba[e], mul2(v[2 + e], bb[e])) : mul2(v[2 + e], bb[e]);
      }
      if (NORM) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = mul2(o[e], r2);
      }
      if (c.h + k * RPW + g < c.end) L.store(y + k * RPW * D, o);
    }
    walk.next(c);
  }
  tc::cp_async_wait<0>();
}

template <int D, bool IL, bool NORM>
__global__ void __launch_bounds__(32 * kWarps, kBwdBlocks) rope_bwd_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kRound * 512;
  extern __shared__ __align__(16) unsigned char ring_all[];
  __shared__ __align__(16) float2 table[kWarps][D / 2];
  const RopeDims& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / LPR;
  unsigned char* ring = ring_all + warp * kAhead * (NORM ? 2 : 1) * STEP;      // per slot: dy, then x
  const Lane<D, IL> L(lane, s.rot, a.inv_freq, table[warp]);
  const Walk<RPW * kRound> walk(a);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  Cursor c{static_cast<int64_t>(blockIdx.x) * kWarps + warp, 0, 0, 0};
  walk.open(c);
  Cursor f = c;
  auto fetch = [&](int slot) {
    if (f.wk < walk.work) {
      const int64_t t = walk.token(f);
      const uint32_t dst = tc::su32(ring + slot * (NORM ? 2 : 1) * STEP);
      fetch_rows<D>(dst, a.dy[f.part] + t * (f.part ? s.Hkv : s.Hq) * D, f, lane);
      if (NORM) fetch_rows<D>(dst + STEP, a.x[f.part] + t * (f.part ? s.ks : s.qs), f, lane);
      walk.next(f);
    }
    tc::cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) fetch(k);
  uint64_t dw[2][4];                                       // Q's and K's weight gradients of the lane's elements
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[0][e] = dw[1][e] = 0;
  int64_t now = -1;                                        // the unit and part that the factors are for
  int now_part = 0;
  uint64_t cs2[2], sn2[2], w2[4];
  for (int slot = 0; c.wk < walk.work; slot = slot + 1 == kAhead ? 0 : slot + 1) {
    const int64_t t = walk.token(c);
    if (c.wk != now || c.part != now_part) {
      if (c.wk != now) {
        L.form(lane, a.pos ? a.pos[t] : static_cast<int>(t % s.N), s.rot_scale);
        float cs[4], sn[4];
        L.factors(cs, sn);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          cs2[k] = tc::pack2(cs[2 * k], cs[2 * k + 1]);
          sn2[k] = tc::pack2(sn[2 * k], sn[2 * k + 1]);
        }
      }
      now = c.wk;
      now_part = c.part;
      if (NORM) {
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = a.w[c.part] ? a.w[c.part][L.element(k)] : 1.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) w2[k] = tc::pack2(w[2 * k], w[2 * k + 1]);
      }
    }
    tc::cp_async_wait<kAhead - 2>();
    __syncwarp();                                          // also: every lane has read the slot fetched next
    fetch(slot == 0 ? kAhead - 1 : slot - 1);
    const unsigned char* rows = ring + slot * (NORM ? 2 : 1) * STEP;
    __nv_bfloat16* y = a.y[c.part] + (t * (c.part ? s.Hkv : s.Hq) + c.h + g) * D;
    uint64_t sum[4] = {0, 0, 0, 0};                        // of the step's g h
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
      if (c.h + k * RPW >= c.end) break;                   // the same for the whole warp
      const bool row = c.h + k * RPW + g < c.end;
      uint64_t v[4], gr[4];
      L.load(rows + (k * RPW + g) * D * 2, v);
#pragma unroll
      for (int e = 0; e < 2; ++e) {                        // turned back: first = c first + s second, second = c second - s first
        const uint64_t ms = mul2(sn2[e], tc::pack2(-1.f, -1.f));
        gr[e] = L.turns ? tc::fma2(v[2 + e], sn2[e], mul2(v[e], cs2[e])) : v[e];
        gr[2 + e] = L.turns ? tc::fma2(v[e], ms, mul2(v[2 + e], cs2[e])) : v[2 + e];
      }
      if (NORM) {
        uint64_t x[4], gw[4];
        L.load(rows + STEP + (k * RPW + g) * D * 2, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) gw[e] = mul2(gr[e], w2[e]);
        const uint64_t q = tc::fma2(x[3], x[3], tc::fma2(x[2], x[2], tc::fma2(x[1], x[1], mul2(x[0], x[0]))));
        const uint64_t d = tc::fma2(x[3], gw[3], tc::fma2(x[2], gw[2], tc::fma2(x[1], gw[1], mul2(x[0], gw[0]))));
        float q0, q1, d0, d1;
        tc::unpack2(q, q0, q1);
        tc::unpack2(d, d0, d1);
        const float r = rsqrtf(row_sum<D>(q0 + q1) * (1.f / D) + s.eps);
        const float m = row_sum<D>(d0 + d1) * (-1.f / D) * r * r * r;
        const uint64_t r2 = tc::pack2(r, r), m2 = tc::pack2(m, m);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (row) sum[e] = tc::fma2(mul2(gr[e], x[e]), r2, sum[e]);
          gr[e] = tc::fma2(x[e], m2, mul2(gw[e], r2));
        }
      }
      if (row) L.store(y + k * RPW * D, gr);
    }
    if (NORM) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (c.part) dw[1][e] = tc::add2(dw[1][e], sum[e]);
        else dw[0][e] = tc::add2(dw[0][e], sum[e]);
      }
    }
    walk.next(c);
  }
  tc::cp_async_wait<0>();
  if (NORM && a.partial) {       // the block's sums: lane groups by shuffles, then warps in order
    __syncthreads();             // the ring's last reads are done
    float(*red)[2][D] = reinterpret_cast<float(*)[2][D]>(ring_all);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) tc::unpack2(dw[part][e], v[2 * e], v[2 * e + 1]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int o = 16; o >= LPR; o >>= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
        if (lane < LPR) red[warp][part][L.element(e)] = v[e];
      }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * D; k += 32 * kWarps) {
      float v = 0.f;
      for (int w = 0; w < kWarps; ++w) v += red[w][k / D][k % D];
      a.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + k] = v;
    }
  }
}

// dw[part][e] = sum over the blocks' partials, in a fixed order: 32 interleaved runs, then those.
// grid: (part, 32 elements).
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* partial, int blocks, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int part = blockIdx.x, lane = threadIdx.x & 31, run = threadIdx.x >> 5, e = blockIdx.y * 32 + lane;
  float v = 0.f;
#pragma unroll 8
  for (int k = run; k < blocks; k += 32) v += partial[(static_cast<int64_t>(k) * 2 + part) * D + e];
  red[run][lane] = v;
  __syncthreads();
  float* out = part ? dwk : dwq;
  if (run == 0 && out) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += red[k][lane];
    out[e] = v;
  }
}

int bwd_blocks(const RopeDims& s) {
  const int64_t need = (static_cast<int64_t>(s.B) * s.N + kWarps - 1) / kWarps;
  return static_cast<int>(std::min<int64_t>(need, win::kPlanSms * kBwdBlocks));
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
    static win::Ready ready;
    constexpr int smem = kWarps * kAhead * kRound * 512;
    if (int e = ready(rope_kernel<D, IL, NORM>, smem)) return e;
    ProfScope ps(st, "qk_norm_rope");
    rope_kernel<D, IL, NORM><<<blocks, 32 * kWarps, smem, st>>>(a);
    return cudaGetLastError();
  }
};

template <int D, bool IL, bool NORM>
struct BwdLaunch {
  static int run(const RopeArgs& a, int blocks, float* dwq, float* dwk, cudaStream_t st) {
    static win::Ready ready;
    constexpr int smem = kWarps * kAhead * kRound * 512 * (NORM ? 2 : 1);
    if (int e = ready(rope_bwd_kernel<D, IL, NORM>, smem)) return e;
    {
      ProfScope ps(st, "qk_norm_rope_bwd");
      rope_bwd_kernel<D, IL, NORM><<<blocks, 32 * kWarps, smem, st>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.partial) return e;
    ProfScope ps(st, "qk_norm_rope_dw");
    rope_dw_kernel<D><<<dim3(2, D / 32), 1024, 0, st>>>(a.partial, blocks, dwq, dwk);
    return cudaGetLastError();
  }
};

RopeArgs make_args(const RopeDims& s, const void* Q, const void* K, const float* inv_freq, const float* wq,
                   const float* wk, const int32_t* pos) {
  RopeArgs a{};
  a.s = s;
  a.heads_per_warp = s.Hq + s.Hkv;
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
  const int64_t room = sm_count() * kFwdBlocks, slots = room * kWarps;
  a.heads_per_warp = a.tokens >= slots ? H : rpw;
  const int64_t work = a.tokens * ((H + a.heads_per_warp - 1) / a.heads_per_warp);
  const int blocks = static_cast<int>(std::min<int64_t>((work + kWarps - 1) / kWarps, room));
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
