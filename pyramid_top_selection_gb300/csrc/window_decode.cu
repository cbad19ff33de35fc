// One decode step of the sliding-window attention with sinks over a rolling key/value cache:
// append and attend, one launch.
//
// o = softmax over the visible keys of (s q.k) times V, per head; bound by HBM: every visible key
// and value is read once (4 d bytes per KV head and key) for the up to 8 query heads of a group.
//
// A cluster of CTAs takes one (sequence, KV head, 8 query heads); each of its warps walks its own
// chunks of 16 keys with its own running maximum, sum and output, so no warp waits for another
// until the end. Keys and values arrive by cp.async (a row each; the cache's rows lie Hkv rows
// apart, and roll over) into the warp's ring of stages. S^T = K Q^T and O^T += V^T P^T on m16n8k16 MMAs:
// with keys (then dims) as the 16 rows, a group's 8 heads are the 8 columns and nothing is padded up
// to 16; P^T goes from accumulator to operand layout by a register transposition. The tcgen05 unit's
// 128-row tiles would be 94 % padding here. Warps join through shared memory, CTAs through the
// cluster's distributed shared memory, in a fixed order: no workspace, no second launch.
// 32 sequences, 32 heads over 8, 4100 keys: 83 us, 6.5 TB/s; one sequence, 16 heads over 2, 1028 keys: 7 us.
#include <algorithm>

#include "device.cuh"
#include "internal.h"
#include "profile.h"
#include "window_tc.cuh"

namespace pisa {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kWarps = 4, kStages = 3, kChunk = 16, kHeads = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;                  // log2 growth of the maximum that O is rescaled for

struct WinDecodeArgs {
  WinDecodeDims s;
  const int32_t* pos;
  bf16 *Kc, *Vc;
  const bf16 *q, *k_new, *v_new;
  bf16* o;
  float* lse;
  int32_t* status;
  int32_t sets;            // sets of 8 heads of a group
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

template <int D>
struct DecodeSmem {
  static constexpr int ROW = D * 2;                              // bytes of a key
  static constexpr int STAGE = 2 * kChunk * ROW;                 // keys, then values
  static constexpr int WARP = kStages * STAGE;
  static constexpr int OUT = kHeads * (D + 2) * 4;               // per warp: O, m, l
  static constexpr int bytes = kWarps * WARP;
  static_assert(WARP >= OUT, "the warp's results fit its stages");
};

// What a running maximum stands for in an exponent: as long as every score was -inf, nothing is to be
// subtracted, and 2^-inf is 0 as it should be.
__device__ __forceinline__ float base_of(float m) { return m > neg_inf() ? m : 0.f; }

// One CTA's results, read by the others of its cluster.
template <int D>
struct Joined {
  float o[kHeads][D], m[kHeads], l[kHeads];
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps) window_decode_kernel(const WinDecodeArgs a, int splits) {
  using M = DecodeSmem<D>;
  constexpr int CH = D / 8, KS = D / 16;                         // 16-byte pieces, MMA steps of a row
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ Joined<D> s_join;
  const WinDecodeDims& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, p2 = lane & 3;
  const int rank = static_cast<int>(win::cluster_rank());
  const int kv = blockIdx.y / a.sets, set = blockIdx.y % a.sets, b = blockIdx.z;
  const int heads = min(kHeads, s.G - set * kHeads), h0 = kv * s.G + set * kHeads;
  const int p = a.pos[b];
  if (p < 0 || (p >= s.Ncap && s.Ncap - s.sinks < s.window)) {   // the whole cluster leaves
    if (rank == 0 && threadIdx.x == 0) atomicOr(a.status, PISA_STATUS_POS_RANGE);
    return;
  }
  // the visible keys as one list: ns sinks, then positions lo .. p, whose slots start at s0 and roll over
  const int ring = s.Ncap - s.sinks;
  int lo = max(0, p - s.window + 1);
  if (lo < s.sinks) lo = 0;
  const int ns = lo ? s.sinks : 0, n = ns + (p - lo + 1);
  const int s0 = lo < s.Ncap ? lo : s.sinks + (lo - s.sinks) % ring;
  auto slot_of = [&](int v) {
    if (v < ns) return v;
    const int x = s0 + (v - ns);
    return x < s.Ncap ? x : x - ring;
  };
  const int64_t row = static_cast<int64_t>(s.Hkv) * D;           // elements between slots
  bf16* Kb = a.Kc + (static_cast<int64_t>(b) * s.Ncap * s.Hkv + kv) * D;
  bf16* Vb = a.Vc + (static_cast<int64_t>(b) * s.Ncap * s.Hkv + kv) * D;
  const bf16* kn = a.k_new + (static_cast<int64_t>(b) * s.Hkv + kv) * D;
  const bf16* vn = a.v_new + (static_cast<int64_t>(b) * s.Hkv + kv) * D;
  if (rank == 0 && set == 0 && warp == 0 && lane < CH) {         // append (nothing reads this slot here)
    const int64_t at = slot_of(n - 1) * row + 8 * lane;
    *reinterpret_cast<uint4*>(Kb + at) = ldg_u4(kn + 8 * lane);
    *reinterpret_cast<uint4*>(Vb + at) = ldg_u4(vn + 8 * lane);
  }

  // ---- this warp's chunks of 16 keys: gw, gw + nw, ...
  const int gw = rank * kWarps + warp, nw = splits * kWarps;
  const int chunks = (n + kChunk - 1) / kChunk, mine = chunks > gw ? (chunks - gw + nw - 1) / nw : 0;
  const uint32_t ring_at = tc::su32(sm) + warp * M::WARP;
  // 16-byte piece c of row r of a stage's keys (values: + 16 rows)
  auto piece = [&](int r, int c) { return r * M::ROW + (((c & ~7) | ((c ^ r) & 7)) << 4); };
  auto fetch = [&](int i) {
    if (i < mine) {
      const int v0 = (gw + i * nw) * kChunk, c = lane % CH;
      const uint32_t dst = ring_at + i % kStages * M::STAGE;
#pragma unroll
      for (int k = 0; k < kChunk * CH / 32; ++k) {
        const int r = k * (32 / CH) + lane / CH, v = v0 + r;
        const bool ok = v < n;
        const int64_t at = ok ? slot_of(v) * row + 8 * c : 0;
        const bool fresh = v == n - 1;                           // the new token, wherever its slot is by now
        tc::cp_async16(dst + piece(r, c), fresh ? kn + 8 * c : Kb + at, ok);
        tc::cp_async16(dst + kChunk * M::ROW + piece(r, c), fresh ? vn + 8 * c : Vb + at, ok);
      }
    }
    tc::cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  uint32_t qf[KS][2];                                            // Q^T: heads as columns
  const bf16* qp = a.q + (static_cast<int64_t>(b) * s.Hq + h0 + g) * D + 2 * p2;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    qf[k][0] = g < heads ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * k)) : 0u;
    qf[k][1] = g < heads ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * k + 8)) : 0u;
  }
  const float c1 = s.scale * kLog2e;
  float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.f, 0.f};        // of heads 2 p2, 2 p2 + 1
  float o[KS][4];                                                // O^T: dims 16 k + g (+ 8), those heads
#pragma unroll
  for (int k = 0; k < KS; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;

  for (int i = 0; i < mine; ++i) {
    tc::cp_async_wait<kStages - 2>();
    __syncwarp();
    const uint32_t at = ring_at + i % kStages * M::STAGE;
    float sc[2][4] = {};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t kf[4];
      ldsm4(kf, at + piece(lane & 15, 2 * k + (lane >> 4)));
      mma_bf16(sc[k & 1], kf, qf[k][0], qf[k][1]);
    }
    const int v0 = (gw + i * nw) * kChunk;
    float x[4];                                                  // keys g (0, 1), g + 8 (2, 3) x two heads
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = v0 + g + (e & 2) * 4 < n ? (sc[0][e] + sc[1][e]) * c1 : neg_inf();
    float top[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
    for (int d = 4; d < 32; d *= 2) {
      top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], d));
      top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], d));
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] + kSlack || top[1] > m[1] + kSlack)) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(m[e], top[e]);
        f[e] = tc::ex2(m[e] - base_of(mn));
        m[e] = mn;
        l[e] *= f[e];
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        o[k][0] *= f[0];
        o[k][1] *= f[1];
        o[k][2] *= f[0];
        o[k][3] *= f[1];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = tc::ex2(x[e] - base_of(m[e & 1]));
    l[0] += x[0] + x[2];
    l[1] += x[1] + x[3];
    const uint32_t b0 = transpose8(pack_bf16(x[0], x[1])), b1 = transpose8(pack_bf16(x[2], x[3]));
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t vf[4];
      ldsm4_trans(vf, at + kChunk * M::ROW + piece((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
      mma_bf16(o[k], vf, b0, b1);
    }
    __syncwarp();                                                // every lane has read the stage fetch() refills next
    fetch(i + kStages - 1);
  }
  tc::cp_async_wait<0>();
#pragma unroll
  for (int d = 4; d < 32; d *= 2) {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
    l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
  }

  // ---- join the warps, then the cluster's CTAs
  __syncwarp();
  float* wo = reinterpret_cast<float*>(sm + warp * M::WARP);     // [8][D], then m[8], l[8]
#pragma unroll
  for (int k = 0; k < KS; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) wo[(2 * p2 + (e & 1)) * D + 16 * k + g + (e & 2) * 4] = o[k][e];
  if (g == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      wo[kHeads * D + 2 * p2 + e] = m[e];
      wo[kHeads * D + kHeads + 2 * p2 + e] = l[e];
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < kHeads * D; x += 32 * kWarps) {
    const int h = x / D;
    float mm = neg_inf(), ll = 0.f, oo = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, reinterpret_cast<const float*>(sm + w * M::WARP)[kHeads * D + h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* r = reinterpret_cast<const float*>(sm + w * M::WARP);
      const float f = tc::ex2(r[kHeads * D + h] - base_of(mm));
      oo += f * r[x];
      ll += f * r[kHeads * D + kHeads + h];
    }
    s_join.o[h][x % D] = oo;
    if (x % D == 0) {
      s_join.m[h] = mm;
      s_join.l[h] = ll;
    }
  }
  win::cluster_sync();
  for (int x = rank * 32 * kWarps + threadIdx.x; x < heads * D; x += splits * 32 * kWarps) {
    const int h = x / D;
    float mm = neg_inf(), ll = 0.f, oo = 0.f;
    for (int c = 0; c < splits; ++c) mm = fmaxf(mm, win::ld_cluster_f(&s_join.m[h], c));
    for (int c = 0; c < splits; ++c) {
      const float f = tc::ex2(win::ld_cluster_f(&s_join.m[h], c) - base_of(mm));
      oo += f * win::ld_cluster_f(&s_join.o[h][x % D], c);
      ll += f * win::ld_cluster_f(&s_join.l[h], c);
    }
    const float out = ll == 0.f ? 0.f : oo / ll;                 // 0: all scores were -inf
    a.o[(static_cast<int64_t>(b) * s.Hq + h0 + h) * D + x % D] = __float2bfloat16_rn(out);
    if (x % D == 0 && a.lse) a.lse[static_cast<int64_t>(b) * s.Hq + h0 + h] = (mm + log2f(ll)) * kLn2;
  }
  win::cluster_sync();                                                // nobody leaves while its results are read
}

template <int D>
int decode_launch(const WinDecodeArgs& a, cudaStream_t st) {
  const WinDecodeDims& s = a.s;
  // CTAs of a cluster: as many as run at one time (two an SM, by their shared memory) with at least a
  // chunk of keys for every warp. At 32 sequences x 8 KV heads and 4100 keys, 1 / 2 / 4 / 8 CTAs a
  // unit took 84 / 92 / 103 / 125 us: a second wave, and the start and join of each CTA, cost more
  // than an uneven first wave. A single sequence is latency, and wants all 8.
  const int64_t units = static_cast<int64_t>(s.B) * s.Hkv * a.sets;
  const int64_t keys = std::min<int64_t>(s.Ncap, static_cast<int64_t>(s.window) + s.sinks);
  int splits = 1;
  while (splits < 8 && units * splits * 2 <= sm_count() * 2 && keys > splits * kWarps * kChunk) splits *= 2;
  static win::Ready ready;
  if (int e = ready(window_decode_kernel<D>, DecodeSmem<D>::bytes)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(splits), static_cast<unsigned>(s.Hkv * a.sets), static_cast<unsigned>(s.B));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = DecodeSmem<D>::bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(splits);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  ProfScope ps(st, "window_decode");
  return cudaLaunchKernelEx(&cfg, window_decode_kernel<D>, a, splits);
}

}  // namespace

int launch_window_decode(const WinDecodeDims& s, const int32_t* pos, void* Kc, void* Vc, const void* q,
                         const void* k_new, const void* v_new, void* o, float* lse, int32_t* status, void* stream) {
  const WinDecodeArgs a{s, pos, static_cast<bf16*>(Kc), static_cast<bf16*>(Vc), static_cast<const bf16*>(q),
                        static_cast<const bf16*>(k_new), static_cast<const bf16*>(v_new), static_cast<bf16*>(o), lse,
                        status, (s.G + kHeads - 1) / kHeads};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return s.d == 128 ? decode_launch<128>(a, st) : decode_launch<64>(a, st);
}

}  // namespace pisa
