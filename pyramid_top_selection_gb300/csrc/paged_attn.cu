// Attention of the last tokens of every sequence over a paged cache in 16 or 4 bits.
//
// o = softmax over the visible keys of the scores times V, per query head; bound by HBM: the cached keys and values of a KV head
// are read once (4 d bytes a token, 1.125 d in 4 bits) for up to 16 rows, heads of the group times drafted tokens. More rows are
// sets of 16, units of their own that read them again at another time: one token of 32 sequences of up to 16384, 32 heads
// over 4, takes 94 us (46 in 4 bits), two drafts 101 (63), four, which are two sets, 180 (107). 32 sequences of up
// to 16384 tokens, 32 heads over 8, d = 128, pages of 64: 172 us in 16 bits (6.48 TB/s), 72 in 4 bits (4.35 TB/s: there each
// of 12 warps an SM issues an instruction every five cycles, 620 for a chunk of 4.6 KB, of which 260 turn and
// scale codes; with 128 registers and 16 warps 76 us, with a ring of four stages 72.6). One sequence of 131072 tokens in 4
// bits, 16 heads over 2: 22.3 us, of 64 tokens 11: two kernels' start, three reads that wait for one another, and the joins.
//
// All chunks of all (sequence, KV head, set of rows) units form one list, which is cut into equal runs, one a warp: lengths
// may differ as they like, the work is the same everywhere. The list follows from the lengths, which only the device
// knows, so every warp finds its own run. A warp walks its run with its own running maximum, sum and output. Units that lie
// wholly in a run are written at once; a run's first and last ones may be parts, which the CTA's warps join (the last through
// shared memory, over the ring; a first that is not the last through the workspace), and a second, small kernel joins what
// crosses CTAs. All sums are in the list's order.
//
// S^T = K Q^T and O^T += V^T P^T on m16n8k16 MMAs with tokens (then channels) as the 16 rows and the rows of the unit (heads
// x drafted tokens) as the 8 or 16 columns; tcgen05's 128-row tiles would be 94 % padding. Keys and values come by cp.async
// into each warp's ring.
//   16 bits: chunks of 16 tokens, fragments by ldmatrix.
//   4 bits: chunks of 32 tokens; codes become halves in registers (a code times its scale is exact in fp16: 2 and 4
//   significant bits), with q brought into fp16's range by a power of two per row, and P held 2^7 larger
//   (down to 2^-31 of the largest). A lane of S's fragments takes 32 channels of its token in a row (16 bytes), which channel goes to
//   which slot of the contraction being free; V's fragments want two tokens of one channel in a register, so the nibbles of
//   two tokens are interleaved before they are converted.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "paged.cuh"
#include "profile.h"
#include "scores.cuh"
#include "window_tc.cuh"

namespace pisa {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;                  // log2 growth of the maximum that O is rescaled for
constexpr int kMaxCtas = 3;                    // CTAs of an SM at most, by registers

struct PagedArgs {
  PagedDims s;
  PagedCache c;
  const int32_t *table, *len;
  const bf16* q;
  const float* slopes;
  bf16* o;
  float* lse;
  int32_t* status;
  int32_t* flags;          // per CTA: PISA_STATUS_POS_RANGE if it met a length or page out of range
  float* part;             // parts of units, [rows][D] O, then m and l: two a CTA for the join, then one a warp for the CTA's own
  int32_t sets, rows;      // sets of rows of a KV head; its rows (group heads x nq)
  int32_t units;           // of a sequence: Hkv * sets
};

template <int D, bool FOUR, int NT>
struct Plan {
  static constexpr int CH = FOUR ? 32 : 16;                        // tokens of a chunk
  static constexpr int ROW = FOUR ? D / 2 : D * 2;                 // bytes of a token
  static constexpr int SROW = FOUR ? D / 16 : 0;                   // of its scales
  static constexpr int HALF = CH * (ROW + SROW);                   // keys with their scales; values follow
  static constexpr int STAGE = 2 * HALF;
  static constexpr int ST = 3;
  static constexpr int RING = ST * STAGE;
  static constexpr int COLS = 8 * NT;                              // rows of a unit
  static constexpr int PARTF = COLS * (D + 2), PART = PARTF * 4;   // a part: O [COLS][D], m, l
  static constexpr int TAIL = PART + 2 * kWarps * COLS * 4;        // the run's last part is laid over the ring, the join's factors behind it
  static constexpr int RINGP = RING > TAIL ? RING : TAIL;
  static constexpr int bytes = kWarps * RINGP;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// Transposes an 8x8 matrix of 16-bit values held by a warp (lane 4 g + p: row g, columns 2 p, 2 p + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Shared memory by address.
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t scales_of(uint32_t two) {      // two e4m3 bytes as halves
  const __half2 v = paged::from_e4m3x2(static_cast<uint16_t>(two));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What a running maximum stands for in an exponent: as long as every score was -inf, nothing is to be subtracted.
__device__ __forceinline__ float base_of(float m) { return m > neg_inf() ? m : 0.f; }

// The list of chunks: sequence b's units (KV heads x sets) one after another, n_chunks(b) each.
template <int CH>
struct List {
  const PagedArgs& a;
  int most;
  __device__ __forceinline__ explicit List(const PagedArgs& args) : a(args), most(args.s.max_pages << args.s.log_page) {}
  __device__ __forceinline__ int tokens(int b) const { return max(0, min(a.len[b], most)); }
  static __device__ __forceinline__ int chunks(int n) { return max(1, (n + CH - 1) / CH); }    // an empty sequence has rows to write, too
  // whole warp: the list's length
  __device__ __forceinline__ int64_t total() const {
    int64_t t = 0;
    for (int b = threadIdx.x & 31; b < a.s.B; b += 32) t += chunks(tokens(b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t * a.units;
  }
  // whole warp: the sequence that place t of the list belongs to, and where its first unit begins
  __device__ __forceinline__ void find(int64_t t, int& b, int64_t& begin) const {
    const int lane = threadIdx.x & 31;
    begin = 0;
    for (int b0 = 0; b0 < a.s.B; b0 += 32) {
      const int64_t mine = b0 + lane < a.s.B ? static_cast<int64_t>(chunks(tokens(b0 + lane))) * a.units : 0;
      int64_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, begin + sum > t);
      if (past) {
        const int k = __ffs(past) - 1;
        b = b0 + k;
        begin += __shfl_sync(0xffffffffu, sum - mine, k);
        return;
      }
      begin += __shfl_sync(0xffffffffu, sum, 31);
    }
    b = a.s.B - 1;               // t is below the total
  }
};

// Runs: `n` of them over `total` places, run w the places [begin(w), begin(w + 1)).
struct Runs {
  int64_t total;
  int n;
  __device__ __forceinline__ Runs(int64_t total_, int most) : total(total_), n(static_cast<int>(min(static_cast<int64_t>(most), total_))) {}
  __device__ __forceinline__ int64_t begin(int w) const {
    if (w >= n) return total;
    if (total < (int64_t(1) << 32) / n) return static_cast<uint32_t>(total) * static_cast<uint32_t>(w) / static_cast<uint32_t>(n);
    return total * w / n;
  }
  __device__ __forceinline__ int of(int64_t t) const { return static_cast<int>(((t + 1) * n - 1) / total); }   // the run that has place t
};

// A place in the list.
template <int CH>
struct Place {
  int b, u, c, n, chunks;        // sequence, unit of it, chunk; the sequence's tokens and chunks of a unit
  __device__ __forceinline__ void next(const List<CH>& l) {
    if (++c < chunks) return;
    c = 0;
    if (++u < l.a.units) return;
    u = 0;
    if (++b < l.a.s.B) {
      n = l.tokens(b);
      chunks = l.chunks(n);
    }
  }
};

// A part of a unit, or none (unit -1): whether it has the unit's first and last chunk, and the CTA's first.
struct Part {
  int unit, head, tail, first;
};

// DRAFTS: more than one token a sequence (a variant of its own, for what only they need cost one token of 32 sequences in 4 bits
// 1.9 of 72 us, although it was not run).
template <int D, bool FOUR, int NT, bool DRAFTS>
__global__ void __launch_bounds__(32 * kWarps, NT == 2 ? 2 : 3) paged_attn_kernel(const PagedArgs a) {
  using M = Plan<D, FOUR, NT>;
  constexpr int CH = M::CH, SUB = CH / 16, KS = D / 16;
  constexpr float kLift = FOUR ? 7.f : 0.f;                        // P is held 2^kLift larger
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ Part s_part[kWarps][2];
  __shared__ int s_bad[kWarps][M::ST], s_flag;
  const PagedDims& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, p2 = lane & 3;
  win::grid_wait();                                                // launched while the kernel before ends
  const List<CH> list(a);
  const Runs runs(list.total(), static_cast<int>(gridDim.x) * kWarps);
  if (blockIdx.x * kWarps >= runs.n) {
    if (threadIdx.x == 0) a.flags[blockIdx.x] = 0;
    win::launch_dependents();
    return;
  }
  if (threadIdx.x == 0) s_flag = 0;
  if (threadIdx.x < 2 * kWarps) s_part[threadIdx.x >> 1][threadIdx.x & 1] = Part{-1, 0, 0, 0};
  __syncthreads();
  unsigned char* ring = sm + warp * M::RINGP;
  auto first_part = [&](int k) { return a.part + (2 * static_cast<int64_t>(gridDim.x) + blockIdx.x * kWarps + k) * M::PARTF; };
  const uint32_t ring_at = tc::su32(ring);
  const int w = static_cast<int>(blockIdx.x) * kWarps + warp;
  const int64_t t0 = runs.begin(w);
  const int mine = static_cast<int>(runs.begin(w + 1) - t0);      // 0 past the last run

  if (mine > 0) {
    Place<CH> con;
    {
      int64_t begin;
      list.find(t0, con.b, begin);
      con.n = list.tokens(con.b);
      con.chunks = list.chunks(con.n);
      const int64_t in = t0 - begin;
      con.u = in < (int64_t(1) << 31) ? static_cast<int>(in) / con.chunks : static_cast<int>(in / con.chunks);
      con.c = static_cast<int>(in - static_cast<int64_t>(con.u) * con.chunks);
    }
    Place<CH> fet = con;
    int ids = 0, ids_b = -1, ids_base = 0, fetched = 0;            // page of token ids_base + 16 lane of sequence ids_b
    // byte offset of 16-byte piece c of a token's row
    auto piece = [&](int r, int c) {
      if (FOUR) return r * M::ROW + (D == 128 ? c ^ ((r >> 1) & 2) : c) * 16;
      return r * M::ROW + (((c & ~7) | ((c ^ r) & 7)) << 4);
    };
    // 16-byte pieces of 16 tokens: a lane's are those at lane + 32 x; rows of a piece's run of 32 lanes
    constexpr int P = M::ROW / 16, NP = P / 2, RPX = 32 / P;
    const int lane_from = lane * 16, lane_to = piece(lane / P, lane % P);
    // a KV head's page in bytes, the pages' distance; where the lane's pieces of page 0 of fet's KV head lie: keys, values and
    // (4 bits) the scales of keys or values
    const uint32_t head_bytes = static_cast<uint32_t>(s.page) * M::ROW, page_bytes = head_bytes * s.Hkv;
    const unsigned char *kp0 = nullptr, *vp0 = nullptr, *sp0 = nullptr;
    const uint32_t lane_scale = CH * M::ROW + (lane >= 16 ? M::HALF : 0) + 16 * (lane & 15);
    uint32_t at_f = ring_at;                                       // the stage that is filled next, and its flag
    int* bad_f = s_bad[warp];
    auto unit_f = [&]() {
      const int64_t head = static_cast<int64_t>(fet.u / a.sets) * head_bytes;
      kp0 = a.c.k + head + lane_from;
      vp0 = a.c.v + head + lane_from;
      if (FOUR) sp0 = (lane >= 16 ? a.c.vs : a.c.ks) + (head >> 3) + 16 * (lane & 15);   // a token's scales: an eighth of its codes
    };
    unit_f();
    auto fetch = [&]() {
      if (fetched < mine) {
        const int v0 = fet.c * CH;
        if (fet.b != ids_b || static_cast<uint32_t>(v0 - ids_base) >= 512u) {
          ids_b = fet.b;
          ids_base = v0 & ~511;
          const int tok = ids_base + 16 * lane, len = a.len[fet.b];
          ids = tok < fet.n ? __ldg(a.table + static_cast<int64_t>(fet.b) * s.max_pages + (tok >> s.log_page)) : 0;
          if (len < 0 || len > list.most) s_flag = 1;
        }
        int bad = 0;
        // `N` 16-token blocks from block k of the chunk on, which lie in one page
        auto blocks = [&](auto first, auto number) {
          constexpr int k = decltype(first)::value, N = decltype(number)::value;
          const int tok = v0 + 16 * k, left = fet.n - tok;
          uint32_t page = __shfl_sync(0xffffffffu, ids, tok >> 4);         // (the lane's number modulo 32)
          const bool known = page < static_cast<uint32_t>(s.n_pages), ok = left > 0 && known;
          if (left > 0 && !known) bad |= ((1 << N) - 1) << k;
          const uint32_t in_page = static_cast<uint32_t>(tok & (s.page - 1)) * M::ROW;
          if constexpr (FOUR) {
            // slots behind the end come along: whatever they hold, their scores are hidden and their scales set to 0
            if (ok) {
              const unsigned char* kp = kp0 + static_cast<uint64_t>(page) * page_bytes + in_page;
              const unsigned char* vp = vp0 + static_cast<uint64_t>(page) * page_bytes + in_page;
              const uint32_t to = at_f + k * 16 * M::ROW + lane_to;
#pragma unroll
              for (int x = 0; x < N * NP; ++x) {
                // (the piece's permutation goes by bit 2 of the row: the same for rows 8 apart)
                static_assert(D == 64 || RPX == 8, "a lane's pieces lie 8 rows apart");
                tc::cp_async16(to + x * 512, kp + x * 512, true);
                tc::cp_async16(to + x * 512 + M::HALF, vp + x * 512, true);
              }
              if ((lane & 15) < N * M::SROW)       // lanes 0 .. take the keys' scales, 16 .. the values'
                tc::cp_async16(at_f + lane_scale + k * 16 * M::SROW, sp0 + static_cast<uint64_t>(page) * (page_bytes >> 3) + (in_page >> 3), true);
            }
          } else {
            if (!ok) page = 0;
            const unsigned char* kp = kp0 + static_cast<uint64_t>(page) * page_bytes + in_page;
            const unsigned char* vp = vp0 + static_cast<uint64_t>(page) * page_bytes + in_page;
#pragma unroll
            for (int x = 0; x < NP; ++x) {
              const int r = x * RPX + lane / P;
              const bool in = ok && r < left;
              const uint32_t dst = at_f + piece(r, lane % P);
              tc::cp_async16(dst, kp + x * 512, in);
              tc::cp_async16(dst + M::HALF, vp + x * 512, in);
            }
          }
        };
        using C0 = std::integral_constant<int, 0>;
        using C1 = std::integral_constant<int, 1>;
        if (SUB == 1) {
          blocks(C0{}, C1{});
        } else if (s.page >= CH) {
          blocks(C0{}, std::integral_constant<int, SUB>{});
        } else {
          blocks(C0{}, C1{});
          blocks(C1{}, C1{});
        }
        if (lane == 0) *bad_f = bad;
        if (bad) s_flag = 1;
        ++fetched;
        at_f += M::STAGE;
        ++bad_f;
        if (at_f == ring_at + M::RING) {
          at_f = ring_at;
          bad_f = s_bad[warp];
        }
        fet.next(list);
        if (fet.c == 0) unit_f();
      }
      tc::cp_async_commit();
    };
#pragma unroll 1                                                   // (code that short runs would wait for)
    for (int i = 0; i < M::ST - 1; ++i) fetch();

    uint32_t qf[NT][KS][2];                                        // Q^T: rows of the unit as columns
    // of columns 2 p2, 2 p2 + 1: what a product is multiplied by, at once (c1) or in the exponent (cz); slope log2 e
    float c1[NT][2], cz[NT][2], slope[NT][2];
    int pos[NT][2];
    float m[NT][2], l[NT][2], o[NT][KS][4];
    int begun = 0;                                                 // the part's first chunk
    auto unit_rows = [&](int u) { return min(M::COLS, a.rows - u % a.sets * M::COLS); };
    // row x of unit u: the offset of its q and o in rows of D, its place in slopes, its position
    auto row_at = [&](const Place<CH>& p, int x) {
      const int r = p.u % a.sets * M::COLS + x, i = r / s.G, h = p.u / a.sets * s.G + r % s.G;
      return (static_cast<int64_t>(p.b) * s.nq + i) * s.Hq + h;
    };
    auto open = [&]() {
      begun = con.c;
      const int rows = unit_rows(con.u), kv = con.u / a.sets;
      const float scale = s.scale * (FOUR && a.c.k_amp ? __ldg(a.c.k_amp + kv) : 1.f) * (s.cap > 0.f ? 1.f / s.cap : kLog2e);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int x = 8 * t + g;
        const bool in = x < rows;
        float up = 1.f;
        if (FOUR) {
          // channels D / 4 p2 ..: a lane's quarter of the row
          const bf16* qp = a.q + (in ? row_at(con, x) : 0) * D + D / 4 * p2;
          uint32_t raw[D / 8];
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint4 v = in ? ldg_u4(qp + 8 * k) : make_uint4(0, 0, 0, 0);
            raw[4 * k] = v.x;
            raw[4 * k + 1] = v.y;
            raw[4 * k + 2] = v.z;
            raw[4 * k + 3] = v.w;
          }
#pragma unroll
          for (int k = 0; k < D / 8; ++k) top = __vmaxu2(top, raw[k] & 0x7fff7fffu);
          top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = max(top & 0xffffu, top >> 16);
          // the largest magnitude between 2^7 and 2^8, by a power of two; its reciprocal goes into the scale
          const int e = min(max(static_cast<int>(top >> 7), 14), 254) - 127 - 7;
          const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t v = raw[2 * k + y];
              qf[t][k][y] = pack_f16(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xffff0000u) * down);
            }
          }
        } else {
          const bf16* qp = a.q + (in ? row_at(con, x) : 0) * D + 2 * p2;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qf[t][k][0] = in ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * k)) : 0u;
            qf[t][k][1] = in ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * k + 8)) : 0u;
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = 8 * t + 2 * p2 + e, r = con.u % a.sets * M::COLS + col;
          const bool there = col < rows;
          c1[t][e] = scale * __shfl_sync(0xffffffffu, up, 8 * p2 + 4 * e);
          // (never 0, which hidden scores of -inf would turn into NaN: a row of zeros takes up = 2^-120, times a small amp)
          cz[t][e] = s.cap > 0.f || a.slopes ? 1.f : c1[t][e] == 0.f ? 0x1p-126f : c1[t][e];
          slope[t][e] = there && a.slopes ? __ldg(a.slopes + kv * s.G + r % s.G) * kLog2e : 0.f;
          pos[t][e] = there ? con.n - s.nq + r / s.G : -1;
          m[t][e] = neg_inf();
          l[t][e] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) o[t][k][0] = o[t][k][1] = o[t][k][2] = o[t][k][3] = 0.f;
      }
    };
    // channel of o[..][k][e]
    auto channel = [&](int k, int e) { return FOUR ? D / 8 * g + 2 * k + (e >> 1) : 16 * k + g + 8 * (e >> 1); };
    // the part at hand is over: the unit's output if it is all of it, else a part; last: of the run
    auto close = [&](bool tail, bool last) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], d);
      const bool head = begun == 0;
      if (head && tail) {
        const int rows = unit_rows(con.u);
        const float amp = FOUR && a.c.v_amp ? __ldg(a.c.v_amp + con.u / a.sets) : 1.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = 8 * t + 2 * p2 + e;
            if (x >= rows) continue;
            const int64_t at = row_at(con, x);
            const float inv = l[t][e] == 0.f ? 0.f : amp / l[t][e];
            if (FOUR) {
              uint32_t v[KS];
#pragma unroll
              for (int k = 0; k < KS; ++k)
                v[k] = l[t][e] == 0.f ? 0u : pack_bf16(o[t][k][e] * inv, o[t][k][e + 2] * inv);
#pragma unroll
              for (int k = 0; k < KS; k += 4)
                *reinterpret_cast<uint4*>(a.o + at * D + D / 8 * g + 2 * k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            } else {
#pragma unroll
              for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  a.o[at * D + channel(k, 2 * y)] = __float2bfloat16_rn(l[t][e] == 0.f ? 0.f : o[t][k][e + 2 * y] * inv);
            }
            if (g == 0 && a.lse) a.lse[at] = l[t][e] == 0.f ? neg_inf() : (m[t][e] - kLift + log2f(l[t][e])) * kLn2;
          }
        return;
      }
      if (last) {                                                  // the run's last part: over the ring, which nothing fills any more
        tc::cp_async_wait<0>();
        __syncwarp();
      }
      float* to = last ? reinterpret_cast<float*>(ring) : first_part(warp);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (FOUR) {                                                // a lane's D / 8 channels lie in a row
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < KS; k += 2)
              *reinterpret_cast<float4*>(to + (8 * t + 2 * p2 + e) * D + channel(k, e)) =
                  make_float4(o[t][k][e], o[t][k][e + 2], o[t][k + 1][e], o[t][k + 1][e + 2]);
        } else {
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) to[(8 * t + 2 * p2 + (e & 1)) * D + channel(k, e)] = o[t][k][e];
        }
        if (g == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            to[M::COLS * D + 8 * t + 2 * p2 + e] = m[t][e];
            to[M::COLS * D + M::COLS + 8 * t + 2 * p2 + e] = l[t][e];
          }
        }
      }
      if (lane == 0) s_part[warp][last] = Part{con.b * a.units + con.u, head, tail, 0};
    };

    const float cap2 = s.cap * kLog2e;
    const int tok_g = FOUR ? (D == 128 ? g ^ ((g >> 1) & 1) : g ^ ((g >> 2) & 1)) : g;   // the token of S's row g
    // 4 bits: a lane's places in a stage, from the tokens' first 8 rows: K's codes of token tok_g, V's of the tokens of slots
    // 2 p2 and 2 p2 + 1, the scales of both
    const int tok_a = D == 128 ? 2 * p2 ^ (p2 & 1) : 2 * p2 ^ (p2 >> 1), tok_b = tok_a ^ 1, v_grp = D == 128 ? g : g >> 1;
    const uint32_t k_codes = D == 128 ? piece(tok_g, p2) : tok_g * M::ROW + 8 * p2,
                   k_scales = CH * M::ROW + tok_g * M::SROW + (D == 128 ? 2 * p2 : p2),
                   va_codes = D == 128 ? piece(tok_a, g >> 1) + 8 * (g & 1) : tok_a * M::ROW + 4 * g,
                   vb_codes = D == 128 ? piece(tok_b, g >> 1) + 8 * (g & 1) : tok_b * M::ROW + 4 * g,
                   va_scales = CH * M::ROW + tok_a * M::SROW + v_grp, vb_scales = CH * M::ROW + tok_b * M::SROW + v_grp;
    int stage = 0;
    for (int done = 0; done < mine;) {         // the run's chunks of one unit
      open();
      const int count = min(con.chunks - con.c, mine - done);
      int v0 = con.c * CH;
      for (int i = 0; i < count; ++i, v0 += CH) {
        tc::cp_async_wait<M::ST - 2>();
        __syncwarp();
        const int bad = s_bad[warp][stage];
        const uint32_t at = ring_at + stage * M::STAGE;
        float x[NT][SUB][4];
#pragma unroll
        for (int k = 0; k < SUB; ++k) {
          float sc[NT][2][4];
          if constexpr (FOUR) {
            // the lane's codes of tokens tok_g (0) and tok_g + 8 (1), and their scales
            uint32_t wd[2][D / 32], s2[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t row = at + (16 * k + 8 * r) * M::ROW + k_codes, srow = at + (16 * k + 8 * r) * M::SROW + k_scales;
              if constexpr (D == 128) {
                const uint4 u = lds128(row);
                wd[r][0] = u.x, wd[r][1] = u.y, wd[r][2] = u.z, wd[r][3] = u.w;
                s2[r] = scales_of(lds16(srow));
              } else {
                const uint2 u = lds64(row);
                wd[r][0] = u.x, wd[r][1] = u.y;
                s2[r] = scales_of(lds8(srow));
              }
            }
#pragma unroll
            for (int grp = 0; grp < D / 64; ++grp) {               // 16 channels: two words of a token's
              const uint32_t f0 = __byte_perm(s2[0], 0, grp ? 0x3232u : 0x1010u), f1 = __byte_perm(s2[1], 0, grp ? 0x3232u : 0x1010u);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t h0[4], h1[4];
                paged::from_e2m1x8(wd[0][2 * grp + h], h0);
                paged::from_e2m1x8(wd[1][2 * grp + h], h1);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t kf[4] = {mul_h2(h0[2 * y], f0), mul_h2(h1[2 * y], f1), mul_h2(h0[2 * y + 1], f0), mul_h2(h1[2 * y + 1], f1)};
                  const int step = 2 * (2 * grp + h) + y;
#pragma unroll
                  for (int t = 0; t < NT; ++t) {
                    if (step < 2) mma_f16_first(sc[t][y], kf, qf[t][step][0], qf[t][step][1]);
                    else mma_f16(sc[t][y], kf, qf[t][step][0], qf[t][step][1]);
                  }
                }
              }
            }
          } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[t][0][e] = sc[t][1][e] = 0.f;
#pragma unroll
            for (int y = 0; y < KS; ++y) {
              uint32_t kf[4];
              ldsm4(kf, at + piece(lane & 15, 2 * y + (lane >> 4)));
#pragma unroll
              for (int t = 0; t < NT; ++t) mma_bf16(sc[t][y & 1], kf, qf[t][y][0], qf[t][y][1]);
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][k][e] = sc[t][0][e] + sc[t][1][e];
        }
        // scores in powers of two; what is not seen
        const bool full = bad == 0 && v0 + CH <= con.n - s.nq + 1;   // every row sees the whole chunk
        if (s.cap > 0.f) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < SUB; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[t][k][e] = cap2 * tanh_of(x[t][k][e] * c1[t][e & 1]);
        }
        if (a.slopes) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < SUB; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[t][k][e] = x[t][k][e] * (s.cap > 0.f ? 1.f : c1[t][e & 1]) - slope[t][e & 1] * static_cast<float>(pos[t][e & 1] - (v0 + 16 * k + tok_g + 8 * (e >> 1)));
        }
        if (!full) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < SUB; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (v0 + 16 * k + tok_g + 8 * (e >> 1) > pos[t][e & 1] || (bad >> k) & 1) x[t][k][e] = neg_inf();
        }
        // the running maximum follows only when a lane's scores outgrow it: then, and no sooner, by the chunk's maximum
        float top[NT][2];
        bool grow = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = fmaxf(x[t][0][e], x[t][0][e + 2]);
#pragma unroll
            for (int k = 1; k < SUB; ++k) v = tc::max3(v, x[t][k][e], x[t][k][e + 2]);
            top[t][e] = v * cz[t][e];
            grow |= top[t][e] > m[t][e] + kSlack;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = top[t][e];
#pragma unroll
              for (int d = 4; d < 32; d *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
              const float mn = fmaxf(m[t][e], v);
              f[e] = tc::ex2(m[t][e] - base_of(mn));
              m[t][e] = mn;
              l[t][e] *= f[e];
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[t][k][0] *= f[0];
              o[t][k][1] *= f[1];
              o[t][k][2] *= f[0];
              o[t][k][3] *= f[1];
            }
          }
        }
#pragma unroll
        for (int k = 0; k < SUB; ++k) {
          uint32_t pb[NT][2];                                        // P^T: tokens x rows
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][k][e] = tc::ex2(fmaf(x[t][k][e], cz[t][e & 1], kLift - base_of(m[t][e & 1])));
            l[t][0] += x[t][k][0] + x[t][k][2];
            l[t][1] += x[t][k][1] + x[t][k][3];
            if (FOUR) {
              pb[t][0] = transpose8(pack_f16(x[t][k][0], x[t][k][1]));
              pb[t][1] = transpose8(pack_f16(x[t][k][2], x[t][k][3]));
            } else {
              pb[t][0] = transpose8(pack_bf16(x[t][k][0], x[t][k][1]));
              pb[t][1] = transpose8(pack_bf16(x[t][k][2], x[t][k][3]));
            }
          }
          // Values that are not finite, of a drafted token that earlier queries do not see: their weights of 0 would make NaN of them. Added
          // here to those that see them, and left out of the product. Bits of `odd`: the 16 tokens, in 4 bits for the lane's group of channels.
          uint32_t odd = 0;
          if (DRAFTS && !full) {
            const int drafted = max(0, con.n - s.nq + 1 - (v0 + 16 * k));        // the first token that not all queries see
            const uint32_t v_at = at + M::HALF + 16 * k * M::ROW;
            if (drafted < 16) {
              if constexpr (FOUR) {
                for (int u = drafted; u < 16; ++u)
                  odd |= static_cast<uint32_t>(v0 + 16 * k + u < con.n && !((bad >> k) & 1) &&
                                               (lds8(at + M::HALF + CH * M::ROW + (16 * k + u) * M::SROW + v_grp) & 0x7fu) == 0x7fu) << u;
              } else {
                bool not_finite = false;
                for (int c = lane >> 4; c < D / 8; c += 2) {
                  const uint4 v = lds128(v_at + piece(lane & 15, c));
                  const uint32_t m = 0x7fff7fffu, top = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
                  not_finite |= (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u;
                }
                const uint32_t b = __ballot_sync(0xffffffffu, not_finite);
                odd = (b | b >> 16) & 0xffffu & ~((1u << drafted) - 1);
              }
            }
#pragma unroll 1
            for (uint32_t left = __reduce_or_sync(0xffffffffu, odd); left; left &= left - 1) {
              const int u = __ffs(left) - 1, row = FOUR ? (D == 128 ? u ^ ((u >> 1) & 1) : u ^ ((u >> 2) & 1)) & 7 : u & 7;   // S's row of token u
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float lo = __shfl_sync(0xffffffffu, x[t][k][e], 4 * row + p2), hi = __shfl_sync(0xffffffffu, x[t][k][e + 2], 4 * row + p2);
                  const float P = u < 8 ? lo : hi;
                  if (v0 + 16 * k + u > pos[t][e]) continue;
#pragma unroll
                  for (int c = 0; c < KS; ++c)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                      float v = __int_as_float(0x7fc00000);
                      if constexpr (!FOUR) {
                        const int ch = 16 * c + g + 8 * y;
                        v = __uint_as_float(lds16(v_at + piece(u, ch >> 3) + 2 * (ch & 7)) << 16);
                      } else if (!((odd >> u) & 1)) {
                        continue;
                      }
                      o[t][c][e + 2 * y] += P * v;
                    }
                }
              if constexpr (!FOUR) {
                __syncwarp();
                for (int c = lane; c < D / 8; c += 32)
                  asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v_at + piece(u, c)), "r"(0) : "memory");
                __syncwarp();
              }
            }
          }
          if constexpr (FOUR) {
            // the lane's codes of the tokens of slots 2 p2 (a) and 2 p2 + 1 (b), and of those 8 slots on
            uint32_t va[2][D / 64], vb[2][D / 64], f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t rows = at + M::HALF + (16 * k + 8 * h) * M::ROW, srows = at + M::HALF + (16 * k + 8 * h) * M::SROW;
              if constexpr (D == 128) {
                const uint2 ua = lds64(rows + va_codes), ub = lds64(rows + vb_codes);
                va[h][0] = ua.x, va[h][1] = ua.y;
                vb[h][0] = ub.x, vb[h][1] = ub.y;
              } else {
                va[h][0] = lds32(rows + va_codes);
                vb[h][0] = lds32(rows + vb_codes);
              }
              uint32_t sa = lds8(srows + va_scales), sb = lds8(srows + vb_scales);
              if (!full) {                                         // what is behind the end, or was not copied
                if (v0 + 16 * k + 8 * h + tok_a >= con.n || (bad >> k) & 1) sa = 0;
                if (v0 + 16 * k + 8 * h + tok_b >= con.n || (bad >> k) & 1) sb = 0;
                if ((odd >> (8 * h + tok_a)) & 1) sa = 0;
                if ((odd >> (8 * h + tok_b)) & 1) sb = 0;
              }
              f[h] = scales_of(sa | sb << 8);
            }
#pragma unroll
            for (int wd = 0; wd < D / 64; ++wd) {
              uint32_t lo[2][4], hi[2][4];                           // even and odd channels, both tokens of a pair
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t ua = va[h][wd], ub = vb[h][wd];
                constexpr uint32_t kLow = 0x0f0f0f0fu;
                paged::from_e2m1x8((ua & kLow) | ((ub << 4) & ~kLow), lo[h]);
                paged::from_e2m1x8(((ua >> 4) & kLow) | (ub & ~kLow), hi[h]);
              }
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t vf[4] = {mul_h2(lo[0][y], f[0]), mul_h2(hi[0][y], f[0]), mul_h2(lo[1][y], f[1]), mul_h2(hi[1][y], f[1])};
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(o[t][4 * wd + y], vf, pb[t][0], pb[t][1]);
              }
            }
          } else {
#pragma unroll
            for (int y = 0; y < KS; ++y) {
              uint32_t vf[4];
              ldsm4_trans(vf, at + M::HALF + piece((lane & 7) + ((lane >> 4) << 3), 2 * y + ((lane >> 3) & 1)));
#pragma unroll
              for (int t = 0; t < NT; ++t) mma_bf16(o[t][y], vf, pb[t][0], pb[t][1]);
            }
          }
        }
        __syncwarp();                                                // every lane has read the stage that fetch() refills next
        fetch();
        stage = stage + 1 == M::ST ? 0 : stage + 1;
      }
      const bool first = warp == 0 && done == 0;                   // the part has the CTA's first chunk
      done += count;
      con.c += count - 1;
      const bool tail = con.c + 1 == con.chunks;
      close(tail, done == mine);
      __syncwarp();
      if (lane == 0 && first && !(begun == 0 && tail)) s_part[warp][done == mine].first = 1;
      con.next(list);
    }
    tc::cp_async_wait<0>();
  }
  __syncthreads();
  if (threadIdx.x == 0) a.flags[blockIdx.x] = s_flag ? PISA_STATUS_POS_RANGE : 0;
  // ---- join the warps' parts: at most two a warp, in the list's order, those of one unit next to one another
  float* f_of = reinterpret_cast<float*>(sm) + M::PARTF;           // [2 kWarps][COLS]: behind the first warp's part, in its ring
  int at = 0;
  while (at < 2 * kWarps) {
    const Part p = s_part[at >> 1][at & 1];
    if (p.unit < 0) {
      ++at;
      continue;
    }
    int end = at + 1;
    bool tail = p.tail;
    uint32_t in = 1u << at;
    for (; end < 2 * kWarps; ++end) {
      const Part x = s_part[end >> 1][end & 1];
      if (x.unit >= 0 && x.unit != p.unit) break;
      if (x.unit == p.unit) {
        tail |= x.tail;
        in |= 1u << end;
      }
    }
    const int b = p.unit / a.units, u = p.unit % a.units, rows = min(M::COLS, a.rows - u % a.sets * M::COLS);
    auto part = [&](int k) -> const float* {
      return k & 1 ? reinterpret_cast<const float*>(sm + (k >> 1) * M::RINGP) : first_part(k >> 1);
    };
    const bool whole = p.head && tail;
    float* to = a.part + (2 * static_cast<int64_t>(blockIdx.x) + (p.first ? 0 : 1)) * M::PARTF;
    const float amp = FOUR && a.c.v_amp ? __ldg(a.c.v_amp + u / a.sets) : 1.f;
    auto row_of = [&](int x) {
      const int r = u % a.sets * M::COLS + x, i = r / s.G, h = u / a.sets * s.G + r % s.G;
      return (static_cast<int64_t>(b) * s.nq + i) * s.Hq + h;
    };
    if (threadIdx.x < rows) {                                      // a row's factor of every part, and its sum
      const int x = threadIdx.x;
      float pm[2 * kWarps], mm = neg_inf(), ll = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * kWarps; ++k) {
        pm[k] = (in >> k) & 1 ? part(k)[M::COLS * D + x] : neg_inf();
        mm = fmaxf(mm, pm[k]);
      }
#pragma unroll
      for (int k = 0; k < 2 * kWarps; ++k) {
        pm[k] = tc::ex2(pm[k] - base_of(mm));
        if ((in >> k) & 1) ll += pm[k] * part(k)[M::COLS * D + M::COLS + x];
      }
      const float inv = !whole ? 1.f : ll == 0.f ? 0.f : amp / ll;
#pragma unroll
      for (int k = 0; k < 2 * kWarps; ++k) f_of[k * M::COLS + x] = pm[k] * inv;
      if (!whole) {
        to[M::COLS * D + x] = mm;
        to[M::COLS * D + M::COLS + x] = ll;
      } else if (a.lse) {
        a.lse[row_of(x)] = ll == 0.f ? neg_inf() : (mm - kLift + log2f(ll)) * kLn2;
      }
    }
    __syncthreads();
    for (int y = threadIdx.x; y < rows * (D / 4); y += 32 * kWarps) {
      const int x = y / (D / 4), e = 4 * (y % (D / 4));
      float4 v[2 * kWarps], oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 2 * kWarps; ++k)
        v[k] = (in >> k) & 1 ? *reinterpret_cast<const float4*>(part(k) + x * D + e) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 2 * kWarps; ++k) {
        const float f = f_of[k * M::COLS + x];
        if ((in >> k) & 1) {
          oo.x += f * v[k].x;
          oo.y += f * v[k].y;
          oo.z += f * v[k].z;
          oo.w += f * v[k].w;
        }
      }
      if (whole) *reinterpret_cast<uint2*>(a.o + row_of(x) * D + e) = make_uint2(pack_bf16(oo.x, oo.y), pack_bf16(oo.z, oo.w));
      else *reinterpret_cast<float4*>(to + x * D + e) = oo;
    }
    __syncthreads();                                               // before the next unit's factors
    at = end;
  }
  win::launch_dependents();
}

// Units that cross CTAs: a block joins one row (blockIdx.y) of one of them. Block x of BY_UNIT takes unit x of all; else, where
// there are more units than CTAs, the unit that crosses into CTA x + 1, if that is the first CTA that it crosses into. Also
// the status word, from the CTAs' flags.
template <int D, bool FOUR, int NT, int THREADS, bool BY_UNIT>
__global__ void __launch_bounds__(THREADS) paged_join_kernel(const PagedArgs a, int ctas) {
  using M = Plan<D, FOUR, NT>;
  constexpr int LPR = D / 4, GR = THREADS / LPR;                   // lanes of a row, parts at a time
  constexpr float kLift = FOUR ? 7.f : 0.f;
  __shared__ float s_m[GR], s_l[GR];
  __shared__ float4 s_o[GR][LPR];
  const PagedDims& s = a.s;
  win::launch_dependents();                                        // (what may start now waits for all of this kernel before it reads or writes)
  const List<M::CH> list(a);
  const Runs runs(list.total(), ctas * kWarps);
  const int x = blockIdx.y, lane = threadIdx.x & 31;
  int b = 0, u = 0, c = 0, last = 0;                               // the unit, and the first and last of its CTAs
  int64_t begin = 0;
  bool mine = true;
  if (BY_UNIT) {
    b = static_cast<int>(blockIdx.x) / a.units;
    u = static_cast<int>(blockIdx.x) % a.units;
    for (int k = lane; k < b; k += 32) begin += list.chunks(list.tokens(k));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) begin += __shfl_xor_sync(0xffffffffu, begin, o);
    begin *= a.units;
  } else {
    c = static_cast<int>(blockIdx.x);
    const int64_t t = runs.begin((c + 1) * kWarps);
    mine = t < runs.total;
    if (mine) {
      list.find(t, b, begin);
      u = static_cast<int>((t - begin) / list.chunks(list.tokens(b)));
    }
  }
  if (mine) {
    const int chunks = list.chunks(list.tokens(b));
    begin += static_cast<int64_t>(u) * chunks;
    const int first = runs.of(begin) / kWarps;
    last = runs.of(begin + chunks - 1) / kWarps;
    mine = first < last && (BY_UNIT || first == c) && x < min(M::COLS, a.rows - u % a.sets * M::COLS);
    c = first;
  }
  // only the first of its CTAs can have begun before the unit
  const int late = mine && runs.begin(c * kWarps) < begin ? c : -1;
  win::grid_wait();
  if (blockIdx.x == 0 && x == 0 && threadIdx.x < 32) {
    int any = 0;
    for (int k = lane; k < ctas; k += 32) any |= a.flags[k];
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) *a.status = any ? PISA_STATUS_POS_RANGE : 0;
  }
  if (!mine) return;
  const int gr = threadIdx.x / LPR, e = threadIdx.x % LPR;
  auto part = [&](int k) { return a.part + (2 * static_cast<int64_t>(k) + (k == late)) * M::PARTF; };
  // eight parts at a time, against their maximum so far
  float mm = neg_inf(), ll = 0.f;
  float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = c + gr; k0 <= last; k0 += 8 * GR) {
    float pm[8], pl[8], top = mm;
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool in = k0 + k * GR <= last;
      const float* p = part(in ? k0 + k * GR : c);
      pm[k] = in ? p[M::COLS * D + x] : neg_inf();
      pl[k] = p[M::COLS * D + M::COLS + x];
      v[k] = *reinterpret_cast<const float4*>(p + x * D + 4 * e);
      top = fmaxf(top, pm[k]);
    }
    const float f0 = tc::ex2(mm - base_of(top));
    mm = top;
    ll *= f0;
    oo.x *= f0;
    oo.y *= f0;
    oo.z *= f0;
    oo.w *= f0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k0 + k * GR > last) continue;                            // no part (a part's NaN goes on, whatever its factor)
      const float f = tc::ex2(pm[k] - base_of(top));
      oo.x += f * v[k].x;
      oo.y += f * v[k].y;
      oo.z += f * v[k].z;
      oo.w += f * v[k].w;
      ll += f * pl[k];
    }
  }
  s_o[gr][e] = oo;
  if (e == 0) {
    s_m[gr] = mm;
    s_l[gr] = ll;
  }
  __syncthreads();
  if (gr > 0) return;
#pragma unroll
  for (int k = 1; k < GR; ++k) mm = fmaxf(mm, s_m[k]);
  ll = 0.f;
  oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < GR; ++k) {
    const float f = tc::ex2(s_m[k] - base_of(mm));
    const float4 v = s_o[k][e];
    oo.x += f * v.x;
    oo.y += f * v.y;
    oo.z += f * v.z;
    oo.w += f * v.w;
    ll += f * s_l[k];
  }
  const int r = u % a.sets * M::COLS + x, i = r / s.G, h = u / a.sets * s.G + r % s.G;
  const int64_t row = (static_cast<int64_t>(b) * s.nq + i) * s.Hq + h;
  const float inv = ll == 0.f ? 0.f : (FOUR && a.c.v_amp ? __ldg(a.c.v_amp + u / a.sets) : 1.f) / ll;
  const uint2 out = ll == 0.f ? make_uint2(0, 0) : make_uint2(pack_bf16(oo.x * inv, oo.y * inv), pack_bf16(oo.z * inv, oo.w * inv));
  *reinterpret_cast<uint2*>(a.o + row * D + 4 * e) = out;
  if (e == 0 && a.lse) a.lse[row] = ll == 0.f ? neg_inf() : (mm - kLift + log2f(ll)) * kLn2;
}

int cols_of(const PagedDims& s) { return s.G * s.nq <= 8 ? 8 : 16; }

template <int D, bool FOUR, int NT, bool DRAFTS>
int attn_launch(PagedArgs& a, cudaStream_t st) {
  using M = Plan<D, FOUR, NT>;
  static win::Ready ready;
  static std::atomic<int> known[64];                               // CTAs an SM holds + 1, per device
  int dev = 0;
  if (int e = ready(paged_attn_kernel<D, FOUR, NT, DRAFTS>, M::bytes)) return e;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  int held = dev < 64 ? known[dev].load(std::memory_order_relaxed) - 1 : -1;
  if (held < 0) {
    if (cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&held, paged_attn_kernel<D, FOUR, NT, DRAFTS>, 32 * kWarps, M::bytes)) return e;
    if (held < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) known[dev].store(held + 1, std::memory_order_relaxed);
  }
  const int ctas = std::min(sm_count() * std::min(held, kMaxCtas), win::kPlanSms * kMaxCtas);
  a.sets = (a.rows + M::COLS - 1) / M::COLS;
  a.units = a.s.Hkv * a.sets;
  {
    ProfScope ps(st, "paged_attn");
    const win::Behind b(dim3(ctas), 32 * kWarps, M::bytes, st);
    const PagedArgs& ca = a;
    if (cudaError_t e = cudaLaunchKernelEx(&b.cfg, paged_attn_kernel<D, FOUR, NT, DRAFTS>, ca)) return e;
  }
  ProfScope ps(st, "paged_join");
  // a unit a block where they are fewer than the CTAs, with more threads where they have many parts each
  const int64_t units = static_cast<int64_t>(a.s.B) * a.units;
  const bool by_unit = units < ctas, many = units * 16 < ctas;
  const win::Behind b(dim3(static_cast<unsigned>(by_unit ? units : std::max(1, ctas - 1)), static_cast<unsigned>(std::min(M::COLS, a.rows))),
                      many ? 512 : 128, 0, st);
  const PagedArgs& ca = a;
  if (many) return cudaLaunchKernelEx(&b.cfg, paged_join_kernel<D, FOUR, NT, 512, true>, ca, ctas);
  if (by_unit) return cudaLaunchKernelEx(&b.cfg, paged_join_kernel<D, FOUR, NT, 128, true>, ca, ctas);
  return cudaLaunchKernelEx(&b.cfg, paged_join_kernel<D, FOUR, NT, 128, false>, ca, ctas);
}

template <int D, bool FOUR>
int by_rows(PagedArgs& a, cudaStream_t st) {
  if (a.s.nq > 1) return cols_of(a.s) == 8 ? attn_launch<D, FOUR, 1, true>(a, st) : attn_launch<D, FOUR, 2, true>(a, st);
  return cols_of(a.s) == 8 ? attn_launch<D, FOUR, 1, false>(a, st) : attn_launch<D, FOUR, 2, false>(a, st);
}

constexpr size_t kFlags = 256, kParts = kFlags + (win::kPlanSms * kMaxCtas * 4 + 255) / 256 * 256;

}  // namespace

size_t paged_attn_ws(const PagedDims& s) {
  return kParts + static_cast<size_t>((2 + kWarps) * win::kPlanSms * kMaxCtas) * cols_of(s) * (s.d + 2) * 4;
}

int launch_paged_attn(const PagedDims& s, const PagedCache& c, const int32_t* table, const int32_t* len, const void* q,
                      const float* slopes, void* o, float* lse, char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  PagedArgs a{};
  a.s = s;
  a.c = c;
  a.table = table;
  a.len = len;
  a.q = static_cast<const bf16*>(q);
  a.slopes = slopes;
  a.o = static_cast<bf16*>(o);
  a.lse = lse;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.flags = reinterpret_cast<int32_t*>(ws + kFlags);
  a.part = reinterpret_cast<float*>(ws + kParts);
  a.rows = s.G * s.nq;
  if (s.d == 128) return s.bits == 4 ? by_rows<128, true>(a, st) : by_rows<128, false>(a, st);
  return s.bits == 4 ? by_rows<64, true>(a, st) : by_rows<64, false>(a, st);
}

}  // namespace pisa
