// Append to a paged cache: norm and rotation of keys (and queries) on the way, pages in 16 or 4 bits.
//
// Per row x of d elements: y = x r w turned by its position, as in qk_rope.cu, rounded to bf16 once (so that a 4-bit
// page holds the codes of the very keys that a 16-bit one would hold). Queries go to Qr; keys, and values as they are, into
// their slots. 4 bits: a group of 16 elements v = y / amp has scale s = e4m3(max |v| / 6), and v's code is the
// e2m1 value nearest to v / s; that quotient is v times 1 / s, corrected by its remainder, so that ties come out as
// ties.
//
// Bound: memory. One warp takes one token and runs over its heads (queries, keys, values) in steps of four rounds of 512
// bytes that arrive by cp.async in the warp's ring, two steps ahead of the arithmetic; the slots of 32 tokens
// of a warp are looked up at once, a lane each. With few tokens the heads are split over warps.
#include <algorithm>

#include "internal.h"
#include "paged.cuh"
#include "profile.h"
#include "rope.cuh"

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

struct AppendArgs {
  PagedDims s;
  RopeDims t;
  PagedCache c;
  const bf16* x[3];              // Q, K, V
  int64_t stride[3];
  int32_t heads[3];              // rows of a token: Hq (0 without queries), Hkv, Hkv
  const float* w[2];
  const float* inv_freq;
  const int32_t *table, *seq, *pos;
  bf16* Qr;
  int32_t* status;
  int32_t heads_per_warp, chunks;
  int64_t tokens;
};

// A warp's place: unit of work (token * chunks + chunk of heads), part (Q, K or V), the step's first head, one past
// the last of the unit's heads in this part.
struct Place {
  int64_t wk;
  int part, h, end;
};

template <int ROWS>
struct Steps {
  const AppendArgs& a;
  int64_t work, step;
  __device__ __forceinline__ Steps(const AppendArgs& args)
      : a(args), work(args.tokens * args.chunks), step(static_cast<int64_t>(gridDim.x) * kWarps) {}
  __device__ __forceinline__ int64_t token(const Place& p) const { return a.chunks == 1 ? p.wk : p.wk / a.chunks; }
  // the part from `part` on that has heads of the unit's, or the next unit
  __device__ __forceinline__ void seek(Place& p) const {
    const int beg = a.chunks == 1 ? 0 : static_cast<int>(p.wk % a.chunks) * a.heads_per_warp, end = beg + a.heads_per_warp;
    int at = 0;
    for (int k = 0; k < 3; ++k) {
      const int lo = max(beg - at, 0), hi = min(end - at, a.heads[k]);
      at += a.heads[k];
      if (k >= p.part && lo < hi) {
        p.part = k;
        p.h = lo;
        p.end = hi;
        return;
      }
    }
    p.wk += step;
    p.part = -1;
  }
  __device__ __forceinline__ void open(Place& p) const {
    p.part = 0;
    seek(p);                     // a unit has heads
  }
  __device__ __forceinline__ void next(Place& p) const {
    p.h += ROWS;
    if (p.h < p.end) return;
    ++p.part;
    seek(p);
    if (p.part < 0) open(p);
  }
};

template <int D, bool IL, bool NORM, bool FOUR>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) append_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kRound * 512, ROWS = RPW * kRound;
  extern __shared__ __align__(16) unsigned char ring_all[];
  __shared__ __align__(16) float2 table[kWarps][D / 2];
  const PagedDims& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / LPR, e = 8 * (lane % LPR);
  unsigned char* ring = ring_all + warp * kAhead * STEP;
  const Lane<D, IL> L(lane, a.t.rot, a.inv_freq, table[warp]);
  const Steps<ROWS> steps(a);
  Place c{static_cast<int64_t>(blockIdx.x) * kWarps + warp, 0, 0, 0};
  steps.open(c);
  Place f = c;
  auto fetch = [&](int slot) {
    if (f.wk < steps.work) {
      const bf16* x = a.x[f.part] + steps.token(f) * a.stride[f.part];
#pragma unroll
      for (int k = 0; k < kRound; ++k) {
        const int r = k * RPW + g;
        if (f.h + r < f.end) tc::cp_async16(tc::su32(ring + slot * STEP) + (r * D + e) * 2, x + static_cast<int64_t>(f.h + r) * D + e, true);
      }
      steps.next(f);
    }
    tc::cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) fetch(k);

  int64_t now = -1, row0 = -1;             // the unit at hand, and its slot's row of KV head 0 (-1: nothing is stored)
  int now_part = -1, unit = -1, p0 = 0;    // units so far; the position
  int64_t lane_row = -1;                   // the same of unit (unit & ~31) + lane
  int lane_pos = 0;
  uint64_t aa[2], ab[2], ba[2], bb[2];     // first = aa first + ab second, second = ba first + bb second
  for (int slot = 0; c.wk < steps.work; slot = slot + 1 == kAhead ? 0 : slot + 1) {
    const int64_t t = steps.token(c);
    if (c.wk != now) {
      if ((++unit & 31) == 0) {            // the slots of this warp's next 32 units
        const int64_t wk = c.wk + lane * steps.step;
        lane_row = -1;
        if (wk < steps.work) {
          const int64_t tk = a.chunks == 1 ? wk : wk / a.chunks;
          const int seq = a.seq ? a.seq[tk] : static_cast<int>(tk / a.t.N);
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
    if (c.part < 2 && row0 >= 0 && (c.wk != now || c.part != now_part)) {
      if (c.wk != now) L.form(lane, p0, a.t.rot_scale);
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
    now = c.wk;
    now_part = c.part;
    tc::cp_async_wait<kAhead - 2>();
    __syncwarp();                                          // also: every lane has read the slot fetched next
    fetch(slot == 0 ? kAhead - 1 : slot - 1);
    unsigned char* rows = ring + slot * STEP;
    if (row0 >= 0) {
      if (c.part < 2) {
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
          if (c.h + k * RPW >= c.end) break;               // the same for the whole warp
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
            o[x] = L.turns ? tc::fma2(v[2 + x], ab[x], mul2(v[x], aa[x])) : mul2(v[x], aa[x]);
            o[2 + x] = L.turns ? tc::fma2(v[x], ba[x], mul2(v[2 + x], bb[x])) : mul2(v[2 + x], bb[x]);
          }
          if (NORM) {
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] = mul2(o[x], r2);
          }
          const int h = c.h + k * RPW + g;
          if (FOUR && c.part == 1) {
            L.store(reinterpret_cast<bf16*>(row), o);      // in place: a lane reads and writes its own elements
          } else if (h < c.end) {
            bf16* to = c.part ? reinterpret_cast<bf16*>(a.c.k) + (row0 + static_cast<int64_t>(h) * s.page) * D
                              : a.Qr + (t * s.Hq + h) * D;
            L.store(to, o);
          }
        }
        if (FOUR && c.part == 1) __syncwarp();
      }
      if (c.part == 2 || (FOUR && c.part == 1)) {
        const bool v_part = c.part == 2;
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
          if (c.h + k * RPW >= c.end) break;
          const int h = c.h + k * RPW + g;
          const bool row = h < c.end;
          const uint4 u = *reinterpret_cast<const uint4*>(rows + ((k * RPW + g) * D + e) * 2);
          const int64_t to = row0 + static_cast<int64_t>(h) * s.page;
          if (!FOUR) {
            if (row) *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.c.v) + to * D + e) = u;
            continue;
          }
          const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
          uint32_t top = 0;                                // the largest magnitude's bits: NaN above infinity above all
#pragma unroll
          for (int x = 0; x < 4; ++x) top = max(top, max(uw[x] & 0x7fffu, (uw[x] >> 16) & 0x7fffu));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          const float* amps = v_part ? a.c.v_amp : a.c.k_amp;
          const float amp = amps && row ? amps[h] : 1.f, ramp = amps ? 1.f / amp : 1.f;
          // v / by, to the last bit but in the rarest cases
          auto over = [](float v, float by, float r) { const float q = v * r; return fmaf(r, fmaf(-q, by, v), q); };
          const float most = __uint_as_float(top << 16);
          const uint32_t s8 = top >= 0x7f80u ? 0x7fu : paged::to_e4m3((amps ? over(most, amp, ramp) : most) / 6.f);
          const float sc = __low2float(paged::from_e4m3x2(static_cast<uint16_t>(s8)));
          const float rs = sc > 0.f ? 1.f / sc : 0.f;      // a scale of 0 or NaN: codes of 0
          float x[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            x[y] = __uint_as_float(y & 1 ? uw[y >> 1] & 0xffff0000u : uw[y >> 1] << 16);
            if (amps) x[y] = over(x[y], amp, ramp);
            x[y] = sc > 0.f ? over(x[y], sc, rs) : copysignf(0.f, x[y]);
          }
          const uint32_t codes = paged::to_e2m1x8(x);
          if (row) {
            *reinterpret_cast<uint32_t*>((v_part ? a.c.v : a.c.k) + to * (D / 2) + e / 2) = codes;
            if ((lane & 1) == 0) (v_part ? a.c.vs : a.c.ks)[to * (D / 16) + e / 16] = static_cast<unsigned char>(s8);
          }
        }
      }
    }
    steps.next(c);
  }
  tc::cp_async_wait<0>();
}

template <int D, bool IL, bool NORM, bool FOUR>
int append_launch(const AppendArgs& a, int blocks, cudaStream_t st) {
  static win::Ready ready;
  constexpr int smem = kWarps * kAhead * kRound * 512;
  if (int e = ready(append_kernel<D, IL, NORM, FOUR>, smem)) return e;
  ProfScope ps(st, "paged_append");
  append_kernel<D, IL, NORM, FOUR><<<blocks, 32 * kWarps, smem, st>>>(a);
  return cudaGetLastError();
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
  a.x[0] = static_cast<const bf16*>(Q);
  a.x[1] = static_cast<const bf16*>(K);
  a.x[2] = static_cast<const bf16*>(V);
  a.stride[0] = t.qs;
  a.stride[1] = t.ks;
  a.stride[2] = vs;
  a.heads[0] = Q ? s.Hq : 0;
  a.heads[1] = a.heads[2] = s.Hkv;
  a.w[0] = wq;
  a.w[1] = wk;
  a.inv_freq = inv_freq;
  a.table = table;
  a.seq = seq;
  a.pos = pos;
  a.Qr = static_cast<bf16*>(Qr);
  a.status = status;
  a.tokens = static_cast<int64_t>(t.B) * t.N;
  // all heads of a token to one warp where the tokens alone fill the GPU's warps; else a warp takes
  // one round of rows
  const int H = a.heads[0] + 2 * s.Hkv;
  const int64_t room = sm_count() * kBlocks;
  a.heads_per_warp = a.tokens >= room * kWarps ? H : 256 / s.d;
  a.chunks = (H + a.heads_per_warp - 1) / a.heads_per_warp;
  const int64_t work = a.tokens * a.chunks;
  const int blocks = static_cast<int>(std::min<int64_t>((work + kWarps - 1) / kWarps, room));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.d == 128) return s.bits == 4 ? by_kind<128, true>(a, blocks, st) : by_kind<128, false>(a, blocks, st);
  return s.bits == 4 ? by_kind<64, true>(a, blocks, st) : by_kind<64, false>(a, blocks, st);
}

}  // namespace pisa
