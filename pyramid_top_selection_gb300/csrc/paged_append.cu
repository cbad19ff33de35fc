// Append to a paged cache: norm and rotation of keys (and queries) on the way, pages in 16 or 4 bits.
//
// Per row x of d elements: y = x r w turned by its position, as in qk_rope.cu, rounded to bf16 once (so that a 4-bit
// page holds the codes of the very keys that a 16-bit one would hold). Queries go to Qr; keys, and values as they are, into
// their slots. 4 bits: a group of 16 elements v = y / amp has scale s = e4m3(max |v| / 6), and v's code is the
// e2m1 value nearest to v / s; that quotient is v times 1 / s, corrected by its remainder, so that ties come out as
// ties.
//
// Bound: memory in 16 bits (49K tokens of 16 heads over 2, d = 128: 82.5 us, 6.07 TB/s); in 4 bits the arithmetic
// (5127 tokens of 32 heads over 8: 34.4 us, 3.2 TB/s, some 180 instructions for two rows, issued in 62 % of the cycles; with 1.4
// tokens a warp, the busiest warps' share is 1.3 times the mean). One warp takes one token and runs over its queries, then its keys and values as one list of rows, in steps
// of four rounds of 512 bytes that arrive by cp.async in the warp's ring, two steps ahead of the arithmetic; the slots
// of 32 tokens of a warp are looked up at once, a lane each. With few tokens a warp takes a step.
#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "profile.h"
#include "rope.cuh"
#include "scores.cuh"

namespace pisa {

namespace {

using bf16 = __nv_bfloat16;
using rope::Lane;
using rope::row_sum;
using win::mul2;

constexpr int kWarps = 8;
constexpr int kBlocks = 3;       // blocks an SM holds, by registers
constexpr int kRound = 4;        // row rounds (512 bytes a warp) of a step
constexpr int kAhead = 3;        // steps in a warp's ring: two in flight, one in use
constexpr int kStart = 2;        // a unit's start, in steps

// v / by from r, nearly 1 / by: the quotient corrected by its remainder, right to the last bit but in the rarest cases, and
// exact where v / by is (so are all ties). Pairs alike. With r = 0 (by = 0): 0.
__device__ __forceinline__ float over(float v, float by, float r) {
  const float q = v * r;
  return fmaf(r, fmaf(-q, by, v), q);
}
__device__ __forceinline__ uint64_t over2(uint64_t v, float by, float r) {
  const uint64_t rr = tc::pack2(r, r), q = mul2(v, rr);
  return tc::fma2(rr, tc::fma2(q, tc::pack2(-by, -by), v), q);
}
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

struct AppendArgs {
  PagedDims s;
  RopeDims t;
  PagedCache c;
  const bf16 *Q, *K, *V;
  int64_t vs;
  const float* w[2];
  const float* inv_freq;
  const int32_t *table, *seq, *pos;
  bf16* Qr;
  int32_t* status;
  int32_t q_steps, steps;        // a token's steps: its queries' (0 without), then its keys' and values'
  int32_t per, parts;            // steps of a unit of work, units of a token
  int32_t units;                 // all tokens' (< 2^31, see the launch: the step to the next one is taken only where there is one)
};

// A step of a token: rows [h, end) of its queries (part 0), or of its keys and values (part 1: row r is key r, or value
// r - Hkv).
struct Place {
  int unit, token;
  int step, end;                 // end: of the unit's steps
};

template <int D, bool IL, bool NORM, bool FOUR>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) append_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kRound * 512, ROWS = RPW * kRound;
  extern __shared__ __align__(16) unsigned char ring_all[];
  __shared__ __align__(16) float2 table[kWarps][D / 2];
  const PagedDims& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / LPR, e = 8 * (lane % LPR);
  win::grid_wait();                                        // launched while the kernel before ends
  win::launch_dependents();
  unsigned char* ring = ring_all + warp * kAhead * STEP;
  const Lane<D, IL> L(lane, a.t.rot, a.inv_freq, table[warp]);
  const int stride = static_cast<int>(gridDim.x) * kWarps;
  auto open = [&](Place& p) {
    p.token = a.parts == 1 ? p.unit : p.unit / a.parts;
    p.step = static_cast<int>(p.unit - p.token * a.parts) * a.per;
    p.end = min(a.steps, p.step + a.per);
  };
  auto next = [&](Place& p) {
    if (++p.step < p.end) return;
    p.unit = p.unit < a.units - stride ? p.unit + stride : a.units;
    open(p);
  };
  Place c{static_cast<int>(blockIdx.x) * kWarps + warp, 0, 0, 0};
  open(c);
  Place f = c;
  auto fetch = [&](int slot) {
    if (f.unit < a.units) {
      const uint32_t to = tc::su32(ring + slot * STEP) + lane * 16;
      if (f.step < a.q_steps) {
        const int h = f.step * ROWS + g;
        const bf16* x = a.Q + static_cast<int64_t>(f.token) * a.t.qs + h * D + e;
#pragma unroll
        for (int k = 0; k < kRound; ++k)
          if (h + k * RPW < s.Hq) tc::cp_async16(to + k * 512, x + k * (RPW * D), true);
      } else {
        const int r = (f.step - a.q_steps) * ROWS + g;
        const bf16* xk = a.K + static_cast<int64_t>(f.token) * a.t.ks + r * D + e;
        const bf16* xv = a.V + static_cast<int64_t>(f.token) * a.vs + (r - s.Hkv) * D + e;
#pragma unroll
        for (int k = 0; k < kRound; ++k)
          if (r + k * RPW < 2 * s.Hkv) tc::cp_async16(to + k * 512, (r + k * RPW < s.Hkv ? xk : xv) + k * (RPW * D), true);
      }
      next(f);
    }
    tc::cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) fetch(k);

  int64_t row0 = -1;                       // the slot's row of KV head 0 (-1: nothing is stored)
  int now = -1, now_part = -1, unit = -1, p0 = 0;    // the unit and part at hand, units so far, the position
  int64_t lane_row = -1;                   // the same of unit (unit & ~31) + lane
  int lane_pos = 0;
  uint64_t aa[2], ab[2], ba[2], bb[2];     // first = aa first + ab second, second = ba first + bb second
  for (int slot = 0; c.unit < a.units; slot = slot + 1 == kAhead ? 0 : slot + 1) {
    const int part = c.step >= a.q_steps;
    if (c.unit != now) {
      if ((++unit & 31) == 0) {            // the slots of this warp's next 32 units
        const int64_t u = c.unit + static_cast<int64_t>(lane) * stride;
        lane_row = -1;
        if (u < a.units) {
          const int tk = a.parts == 1 ? static_cast<int>(u) : static_cast<int>(u) / a.parts;
          const int seq = a.seq ? a.seq[tk] : tk / a.t.N;
          lane_pos = a.pos[tk];
          if (seq >= 0) {
            int page = -1;
            if (seq < s.B && lane_pos >= 0 && lane_pos < s.max_pages << s.log_page)
              page = a.table[static_cast<int64_t>(seq) * s.max_pages + (lane_pos >> s.log_page)];
            if (page >= 0 && page < s.n_pages)
              lane_row = static_cast<int64_t>(page) * s.Hkv * s.page + (lane_pos & (s.page - 1));
            else
              atomicOr(a.status, PISA_STATUS_POS_RANGE);
          }
        }
      }
      row0 = __shfl_sync(0xffffffffu, lane_row, unit & 31);
      p0 = __shfl_sync(0xffffffffu, lane_pos, unit & 31);
    }
    if (row0 >= 0 && (c.unit != now || part != now_part)) {
      if (c.unit != now) L.form(lane, p0, a.t.rot_scale);
      float cs[4], sn[4], w[8];
      L.factors(cs, sn);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = NORM && a.w[part] ? a.w[part][L.element(k)] : 1.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        aa[k] = tc::pack2(w[2 * k] * cs[2 * k], w[2 * k + 1] * cs[2 * k + 1]);
        ab[k] = tc::pack2(-w[4 + 2 * k] * sn[2 * k], -w[5 + 2 * k] * sn[2 * k + 1]);
        ba[k] = tc::pack2(w[2 * k] * sn[2 * k], w[2 * k + 1] * sn[2 * k + 1]);
        bb[k] = tc::pack2(w[4 + 2 * k] * cs[2 * k], w[5 + 2 * k] * cs[2 * k + 1]);
      }
    }
    now = c.unit;
    now_part = part;
    tc::cp_async_wait<kAhead - 2>();
    __syncwarp();                                          // also: every lane has read the slot fetched next
    fetch(slot == 0 ? kAhead - 1 : slot - 1);
    unsigned char* rows = ring + slot * STEP;
    const int h0 = (part ? c.step - a.q_steps : c.step) * ROWS, end = part ? 2 * s.Hkv : s.Hq;
    if (row0 >= 0) {
      // where the lane group's first row goes, and from one round's rows to the next's
      bf16* out = part ? reinterpret_cast<bf16*>(a.c.k) + (row0 + static_cast<int64_t>(h0 + g) * s.page) * D
                       : a.Qr + (static_cast<int64_t>(c.token) * s.Hq + h0 + g) * D;
      const int out_step = (part ? s.page : 1) * (RPW * D);
#pragma unroll
      for (int k = 0; k < kRound; ++k) {
        const int h = h0 + k * RPW;
        if (h >= (part ? s.Hkv : end)) break;              // the same for the whole warp
        unsigned char* row = rows + (k * RPW + g) * D * 2;
        uint64_t v[4], o[4];
        L.load(row, v);
        uint64_t r2 = 0;
        if (NORM) {
          const uint64_t q = tc::fma2(v[3], v[3], tc::fma2(v[2], v[2], tc::fma2(v[1], v[1], mul2(v[0], v[0]))));
          float q0, q1;
          tc::unpack2(q, q0, q1);
          const float r = rsqrtf(row_sum<D>(q0 + q1) * (1.f / D) + a.t.eps);
          r2 = tc::pack2(r, r);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          o[x] = mul2(v[x], aa[x]);
          o[2 + x] = mul2(v[2 + x], bb[x]);
        }
        if (L.turns) {                                     // what does not turn does not meet its partner: an infinity there stays itself
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            o[x] = tc::fma2(v[2 + x], ab[x], o[x]);
            o[2 + x] = tc::fma2(v[x], ba[x], o[2 + x]);
          }
        }
        if (NORM) {
#pragma unroll
          for (int x = 0; x < 4; ++x) o[x] = mul2(o[x], r2);
        }
        if (h + g < (part ? s.Hkv : end)) {
          // keys of 4-bit pages go back to the ring, in place: a lane reads and writes its own elements
          L.store(FOUR && part ? reinterpret_cast<bf16*>(row) : out, o);
        }
        out += out_step;
      }
      if (part && FOUR) __syncwarp();
      if (part) {
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
          const int r = h0 + k * RPW + g;
          if (h0 + k * RPW >= end) break;
          if (!FOUR && h0 + (k + 1) * RPW <= s.Hkv) continue;
          const bool value = r >= s.Hkv, in = r < end;
          const int h = value ? r - s.Hkv : r;
          const uint4 u = *reinterpret_cast<const uint4*>(rows + ((k * RPW + g) * D + e) * 2);
          const int64_t to = row0 + static_cast<int64_t>(h) * s.page;
          if (!FOUR) {
            if (in && value) *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.c.v) + to * D + e) = u;
            continue;
          }
          uint32_t uw[4] = {u.x, u.y, u.z, u.w};
          // the largest magnitude's bits: NaN above infinity above all
          uint32_t top = max16x2(max16x2(uw[0] & 0x7fff7fffu, uw[1] & 0x7fff7fffu), max16x2(uw[2] & 0x7fff7fffu, uw[3] & 0x7fff7fffu));
          top = max(top & 0xffffu, top >> 16);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          const float* amps = value ? a.c.v_amp : a.c.k_amp;
          const float amp = amps && in ? amps[h] : 1.f, ramp = rcp_approx(amp);
          // quotients past 4096 all are the largest code (6) of the largest scale (448): they stop there, not at an infinity, which
          // the remainder would turn into NaN
          const uint32_t far = (__float_as_uint(amp) + (12u << 23)) >> 16;
          const bool bad = top >= 0x7f80u;
          if (top > far) {
            top = far;
#pragma unroll
            for (int y = 0; y < 4; ++y) uw[y] = (uw[y] & 0x80008000u) | __vminu2(uw[y] & 0x7fff7fffu, far * 0x10001u);
          }
          const float most = __uint_as_float(top << 16);
          const uint32_t s8 = bad ? 0x7fu : paged::to_e4m3(over(amps ? over(most, amp, ramp) : most, 6.f, 1.f / 6.f));
          const float sc = __low2float(paged::from_e4m3x2(static_cast<uint16_t>(s8)));
          const float rs = sc > 0.f ? rcp_approx(sc) : 0.f;      // a scale of 0: codes of 0 (of NaN: whatever, they stand for NaN)
          float x[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint64_t v = tc::pack2(__uint_as_float(uw[y] << 16), __uint_as_float(uw[y] & 0xffff0000u));
            if (amps) v = over2(v, amp, ramp);
            tc::unpack2(over2(v, sc, rs), x[2 * y], x[2 * y + 1]);
            x[2 * y] = copysignf(x[2 * y], __uint_as_float(uw[y] << 16));          // (a zero's)
            x[2 * y + 1] = copysignf(x[2 * y + 1], __uint_as_float(uw[y]));
          }
          const uint32_t codes = paged::to_e2m1x8(x);
          if (in) {
            *reinterpret_cast<uint32_t*>((value ? a.c.v : a.c.k) + to * (D / 2) + e / 2) = codes;
            if ((lane & 1) == 0) (value ? a.c.vs : a.c.ks)[to * (D / 16) + e / 16] = static_cast<unsigned char>(s8);
          }
        }
      }
    }
    next(c);
  }
  tc::cp_async_wait<0>();
}

template <int D, bool IL, bool NORM, bool FOUR>
int append_launch(const AppendArgs& a, int blocks, cudaStream_t st) {
  static win::Ready ready;
  constexpr int smem = kWarps * kAhead * kRound * 512;
  if (int e = ready(append_kernel<D, IL, NORM, FOUR>, smem)) return e;
  ProfScope ps(st, "paged_append");
  const win::Behind b(dim3(blocks), 32 * kWarps, smem, st);
  return cudaLaunchKernelEx(&b.cfg, append_kernel<D, IL, NORM, FOUR>, a);
}

template <int D, bool FOUR>
int by_kind(const AppendArgs& a, int blocks, cudaStream_t st) {
  if (a.t.interleaved) return a.t.norm ? append_launch<D, true, true, FOUR>(a, blocks, st) : append_launch<D, true, false, FOUR>(a, blocks, st);
  return a.t.norm ? append_launch<D, false, true, FOUR>(a, blocks, st) : append_launch<D, false, false, FOUR>(a, blocks, st);
}

}  // namespace

int launch_paged_append(const PagedDims& s, const PagedCache& c, const RopeDims& t, const void* Q, const void* K,
                        const void* V, int64_t vs, const float* inv_freq, const float* wq, const float* wk,
                        const int32_t* table, const int32_t* seq, const int32_t* pos, void* Qr, int32_t* status,
                        void* stream) {
  AppendArgs a{};
  a.s = s;
  a.t = t;
  a.c = c;
  a.Q = static_cast<const bf16*>(Q);
  a.K = static_cast<const bf16*>(K);
  a.V = static_cast<const bf16*>(V);
  a.vs = vs;
  a.w[0] = wq;
  a.w[1] = wk;
  a.inv_freq = inv_freq;
  a.table = table;
  a.seq = seq;
  a.pos = pos;
  a.Qr = static_cast<bf16*>(Qr);
  a.status = status;
  const int rows = 256 / s.d * kRound;
  const int64_t room = sm_count() * kBlocks, tokens = static_cast<int64_t>(t.B) * t.N;
  a.q_steps = Q ? (s.Hq + rows - 1) / rows : 0;
  a.steps = a.q_steps + (2 * s.Hkv + rows - 1) / rows;
  // A unit of work, which forms its token's angles and looks its slot up (kStart steps' time), is a token's steps or a
  // part of them, whichever has the busiest warp done first (5127 tokens of 32 heads over 8, 6 steps each: 34.0 us with 3 steps
  // a unit, 34.7 with 6, 43.7 with 1).
  const int64_t slots = room * kWarps;
  int64_t least = INT64_MAX;
  for (int parts = 1; parts <= a.steps; ++parts) {
    const int per = (a.steps + parts - 1) / parts;
    const int64_t cost = ((tokens * parts + slots - 1) / slots) * (per + kStart);
    if (cost >= least) continue;
    least = cost;
    a.per = per;
    a.parts = (a.steps + per - 1) / per;
  }
  a.units = static_cast<int>(tokens * a.parts);          // parts <= steps < Hq + 2 Hkv (a step of queries holds one at least, one of keys and values two), and T (Hq + 2 Hkv) < 2^31
  const int blocks = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(a.units) + kWarps - 1) / kWarps, room));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.d == 128) return s.bits == 4 ? by_kind<128, true>(a, blocks, st) : by_kind<128, false>(a, blocks, st);
  return s.bits == 4 ? by_kind<64, true>(a, blocks, st) : by_kind<64, false>(a, blocks, st);
}

}  // namespace pisa
