// What the window attention's kernels share: bounded waits that sleep, register moves between warpgroups,
// the walk over a query tile's keys, clusters, and tensor-core products from descriptors.
#pragma once

#include "tc.cuh"
#include "tmap.h"
#include "window.h"

namespace pisa {
namespace win {

// Wait for the phase of `bar` with this parity: sleeps in try_wait, gives up (and sets the CTA's
// abort flag) after limit_ns nanoseconds, or at once when the CTA has aborted.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort_flag, uint64_t limit_ns) {
  const uint32_t a = tc::su32(bar);
  uint64_t t0 = 0;
  for (int it = 0;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    if (it == 0) t0 = tc::global_ns();
    if ((it & 15) == 15) {
      if (*reinterpret_cast<volatile int*>(abort_flag)) return false;
      if (tc::global_ns() - t0 > limit_ns) break;
    }
  }
  atomicOr(abort_flag, 1);
  return false;
}

// Packed pairs of fp32 (tc.cuh).
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  return tc::fma2(b, tc::pack2(-1.f, -1.f), a);
}

// A value that is the same in the whole warp, in a form that the compiler knows to be: what an MMA
// warp's operands and branches come from then stays in uniform registers (the forward at the 64K prefill
// took 1.60 ms without and 1.44 ms with them).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// TMA store of a shared-memory box into a 4-D tensor map at (c0, c1, c2, c3); what lies outside the
// tensor is not written.
__device__ __forceinline__ void tma_store4(const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
               : "memory");
}

// Bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(tc::su32(bar))
               : "memory");
}

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Heads of a group that share a 128-row tile: the largest power of two dividing G, at most 16. A
// tile's rows are (token, head), heads fastest, so it covers 128 / P tokens and keys are read
// once for its P heads; fewer tokens a tile also means fewer masked keys at a window's edges.
inline int packed_heads(int G) {
  int p = 1;
  while (p < 16 && G % (2 * p) == 0) p *= 2;
  return p;
}

inline int log2_of(int p) {
  int l = 0;
  while (1 << l < p) ++l;
  return l;
}

// Among four neighbouring lanes: lane l's piece c becomes lane c's piece l (16-byte pieces).
__device__ __forceinline__ void transpose4(uint32_t (&u)[4][4], int lane) {
#pragma unroll
  for (int m = 1; m < 4; m *= 2) {
    const bool up = lane & m;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & m) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t t = __shfl_xor_sync(0xffffffffu, up ? u[c][k] : u[c | m][k], m);
        if (up) u[c][k] = t; else u[c | m][k] = t;
      }
    }
  }
}

// Tensor map of [B, N, H, d] bf16 with `stride` elements between tokens: boxes of 64 elements x
// `heads` x `tokens`.
inline int token_map(CUtensorMap* m, const void* p, int B, int N, int H, int d, int64_t stride, int heads, int tokens) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(H), static_cast<uint64_t>(N),
                            static_cast<uint64_t>(B)};
  const uint64_t strides[3] = {static_cast<uint64_t>(d) * 2, static_cast<uint64_t>(stride) * 2,
                               static_cast<uint64_t>(stride) * 2 * N};
  const uint32_t box[4] = {64, static_cast<uint32_t>(heads), static_cast<uint32_t>(tokens), 1};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides, box);
}

// Bits a .. b (inclusive, any integers) of a 32-bit mask.
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  const uint32_t up = b < 0 ? 0u : b >= 31 ? 0xffffffffu : (2u << b) - 1;
  const uint32_t lo = a <= 0 ? 0xffffffffu : a >= 32 ? 0u : ~((1u << a) - 1);
  return up & lo;
}

// Valid tokens of sequence b.
__device__ __forceinline__ int valid_len(const int32_t* len, int b, int N) {
  return len ? max(0, min(__ldg(len + b), N)) : N;
}

// The keys of a run of query positions [p0, p1) of one sequence as one list of columns: first the
// sinks (padded to SP columns, a multiple of 32) when all of these lie before the window's first
// key, then keys lo ... Column v holds key v (v < SP) or lo + v - SP. Otherwise the list simply
// starts at key 0. So every padding column holds a key below lo, one of the sequence's.
struct KeyList {
  int lo, SP, n_cols;
  __device__ __forceinline__ KeyList(int lo_, int SP_) : lo(lo_), SP(SP_), n_cols(0) {}
  __device__ __forceinline__ KeyList(const WinDims& s, int L, int p0, int p1) {
    const int last = min(p1, L) - 1;
    lo = max(0, p0 - s.window + 1);
    SP = (s.sinks + 31) & ~31;
    if (lo < SP) lo = SP = 0;
    n_cols = last >= p0 ? SP + last - lo + 1 : 0;
  }
  __device__ __forceinline__ int key(int v) const { return v < SP ? v : lo + v - SP; }
};

// The 128-column tiles of a key list that hold a key some position in [p0, p1) sees are those from `first` to
// `last`, and those of the sinks before them.
struct TileRange {
  int first, last;
  __device__ __forceinline__ TileRange(const WinDims& s, const KeyList& kl, int L, int p0, int p1) {
    const int end = min(p1, L) - 1;
    last = end < p0 ? -1 : (kl.SP + end - kl.lo) >> 7;
    first = (kl.SP + max(kl.lo, p0 - s.window + 1) - kl.lo) >> 7;
  }
};

// A work item as its CTA's roles take it: decoded by one warp, ahead of the others (the divisions would
// sit at every item's start otherwise), and handed over through a ring in shared memory. n: key tiles of
// 128 columns, -1 past the last item. first / last: the key tiles of the item's row tiles (TileRange).
struct __align__(16) Item {
  int b, kv, h0, t0;
  int L, lo, SP, n;
  int first[2], last[2];
};

constexpr int kItems = 4;

// The CTA's k-th item of n, or -1: rounds of one item a CTA, every second one backwards. Items come
// with the longest first, and a round's first CTA would otherwise always have the longest.
__device__ __forceinline__ int64_t item_of(int k, int n) {
  const int64_t w = static_cast<int64_t>(k) * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  return w < n ? w : -1;
}
__device__ __forceinline__ int rounds_of(int n) { return static_cast<int>((n + static_cast<int64_t>(gridDim.x) - 1) / gridDim.x); }

struct ItemRing {
  Item item[kItems];
  uint64_t full[kItems], empty[kItems];
};

__device__ __forceinline__ void ring_init(ItemRing& q, int consumer_warps) {
  for (int k = 0; k < kItems; ++k) {
    tc::bar_init(&q.full[k], 1);
    tc::bar_init(&q.empty[k], consumer_warps);
  }
}

// Publisher (one lane): item k of the CTA.
__device__ __forceinline__ bool ring_put(ItemRing& q, int k, const Item& it, int* abort_flag, uint64_t limit_ns) {
  if (!wait(&q.empty[k % kItems], ((k / kItems) & 1) ^ 1, abort_flag, limit_ns)) return false;
  q.item[k % kItems] = it;
  tc::bar_arrive(&q.full[k % kItems]);
  return true;
}

// Consumer warp: item k; n = -1 past the last one, or when the CTA gives up.
__device__ __forceinline__ Item ring_get(ItemRing& q, int k, int* abort_flag, uint64_t limit_ns) {
  const bool ok = __all_sync(0xffffffffu, wait(&q.full[k % kItems], (k / kItems) & 1, abort_flag, limit_ns));
  Item it = q.item[k % kItems];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::bar_arrive(&q.empty[k % kItems]);
  if (!ok) it.n = -1;
  it.n = uniform(it.n);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.first[t] = uniform(it.first[t]);
    it.last[t] = uniform(it.last[t]);
  }
  return it;
}

// Clusters: this CTA's number, a barrier over all threads of all its CTAs, and reads of a shared
// variable as CTA `rank` has it.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::su32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f(const float* p, uint32_t rank) {
  return __uint_as_float(ld_cluster_u32(p, rank));
}
__device__ __forceinline__ float2 ld_cluster_f2(const void* p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(const void* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr(p, rank))
               : "memory");
  return v;
}

// Programmatic launches: lets the kernel behind this one start once all CTAs have come here (its CTAs
// take the SMs as they fall free); waits for the kernel before to be complete and its writes visible.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Shared-memory matrix descriptors by their low word (address, MN stride), the part that changes: an
// MMA's operands then cost one addition each to form (tc.cuh has the fields). In a cluster an address
// carries the CTA's number above its 18 bits of offset.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr & 0x3ffff) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn_lo(uint32_t saddr, uint32_t mn_stride) { return ((saddr & 0x3ffff) >> 4) | ((mn_stride >> 4) << 16); }

__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\nsetp.ne.b32 p, %4, 0;\nmov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHigh));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 b;\nsetp.ne.b32 p, %4, 0;\nmov.b64 b, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHigh));
}

// D (128 x 128) = A (128 x DIM) B (128 x DIM)^T, both K-major SW128 tiles (blocks of 64 columns).
template <int DIM>
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo) {
  constexpr uint32_t id = tc::idesc_bf16(128, 128);
#pragma unroll
  for (int k = 0; k < DIM / 16; ++k) {
    const uint32_t o = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
    mma(d, a_lo + o, b_lo + o, id, k > 0);
  }
}

// D (128 x DIM) (+)= A (128 x 128, bf16 in tensor memory) B (128 x DIM), B's rows as stored (MN-major).
// A's columns lie in groups of RUN, each packed in the first half of the RUN 32-bit columns that held the
// fp32 values it was made from.
template <int DIM, int RUN>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, bool accumulate) {
  constexpr uint32_t id = tc::idesc_bf16_major(128, DIM, false, true);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    mma_ts(d, a_tmem + 16 * k / RUN * RUN + 16 * k % RUN / 2, b_lo + k * (2048 >> 4), id, accumulate || k > 0);
}

}  // namespace win
}  // namespace pisa
