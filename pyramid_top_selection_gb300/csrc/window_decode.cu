// One decode step of the sliding-window attention with sinks over a rolling key/value cache:
// append and attend, one warp per (sequence, query head).
#include "device.cuh"
#include "profile.h"
#include "window.h"

namespace pisa {

namespace {

using bf16 = __nv_bfloat16;

struct WinDecodeArgs {
  WinDecodeDims s;
  const int32_t* pos;
  bf16 *Kc, *Vc;
  const bf16 *q, *k_new, *v_new;
  bf16* o;
  float* lse;
  int32_t* status;
};

template <int D>
__global__ void __launch_bounds__(32) window_decode_kernel(const WinDecodeArgs a) {
  constexpr int E = D / 32;
  const WinDecodeDims& s = a.s;
  const int h = blockIdx.x, b = blockIdx.y, kv = h / s.G, lane = threadIdx.x;
  const int p = a.pos[b];
  if (p < 0 || (p >= s.Ncap && s.Ncap - s.sinks < s.window)) {
    if (lane == 0) atomicOr(a.status, PISA_STATUS_POS_RANGE);
    return;
  }
  const int ring = s.Ncap - s.sinks;
  auto slot = [&](int j) -> int64_t { return (j < s.sinks ? j : s.sinks + (j - s.sinks) % ring) + static_cast<int64_t>(b) * s.Ncap; };
  float q[E], o[E] = {}, m = neg_inf(), l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[(static_cast<int64_t>(b) * s.Hq + h) * D + lane * E + e]) * s.scale;
  const bf16* kn = a.k_new + (static_cast<int64_t>(b) * s.Hkv + kv) * D + lane * E;
  const bf16* vn = a.v_new + (static_cast<int64_t>(b) * s.Hkv + kv) * D + lane * E;
  if (h % s.G == 0)
    for (int e = 0; e < E; ++e) {
      a.Kc[(slot(p) * s.Hkv + kv) * D + lane * E + e] = kn[e];
      a.Vc[(slot(p) * s.Hkv + kv) * D + lane * E + e] = vn[e];
    }
  auto key = [&](int j) {
    const int64_t kr = (slot(j) * s.Hkv + kv) * D + lane * E;
    const bf16* k = j == p ? kn : a.Kc + kr;
    const bf16* v = j == p ? vn : a.Vc + kr;
    float x = 0.f;
    for (int e = 0; e < E; ++e) x += q[e] * __bfloat162float(k[e]);
    x = warp_sum(x);
    const float mn = fmaxf(m, x), c = __expf(m - mn), w = __expf(x - mn);
    l = l * c + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * __bfloat162float(v[e]);
    m = mn;
  };
  const int lo = max(0, p - s.window + 1);
  for (int j = 0; j < min(s.sinks, lo); ++j) key(j);
  for (int j = lo; j <= p; ++j) key(j);
  for (int e = 0; e < E; ++e) a.o[(static_cast<int64_t>(b) * s.Hq + h) * D + lane * E + e] = __float2bfloat16_rn(o[e] / l);
  if (lane == 0 && a.lse) a.lse[static_cast<int64_t>(b) * s.Hq + h] = m + logf(l);
}

}  // namespace

int launch_window_decode(const WinDecodeDims& s, const int32_t* pos, void* Kc, void* Vc, const void* q,
                         const void* k_new, const void* v_new, void* o, float* lse, int32_t* status, void* stream) {
  const WinDecodeArgs a{s, pos, static_cast<bf16*>(Kc), static_cast<bf16*>(Vc), static_cast<const bf16*>(q),
                        static_cast<const bf16*>(k_new), static_cast<const bf16*>(v_new), static_cast<bf16*>(o), lse, status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope ps(st, "window_decode");
  (s.d == 128 ? window_decode_kernel<128> : window_decode_kernel<64>)
      <<<dim3(static_cast<unsigned>(s.Hq), static_cast<unsigned>(s.B)), 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pisa
