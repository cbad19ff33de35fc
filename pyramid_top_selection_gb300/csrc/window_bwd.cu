// Sliding-window attention with sinks, backward: sizes and launches of window_bwd.cuh's kernels.
#include <algorithm>

#include "internal.h"
#include "profile.h"
#include "tmap.h"
#include "window_bwd.cuh"

namespace pisa {

size_t align256(size_t x);

namespace {

template <int D>
int bwd_launch(const BwdArgs& a, const CUtensorMap* m, cudaStream_t st) {
  static win::Ready dq_ready, dkv_ready;
  if (int e = dq_ready(window_dq_kernel<D, win::kWindow, 2>, DqSmem<D>::bytes)) return e;
  if (int e = dkv_ready(window_dkv_kernel<D, win::kWindow, 2>, DkvSmem<D>::bytes)) return e;
  const int dq_ctas = std::min({a.n_items, sm_count(), kDqCtas});
  {
    ProfScope ps(st, "window_dq");
    window_dq_kernel<D, win::kWindow, 2><<<dq_ctas, bwd_threads(2), DqSmem<D>::bytes, st>>>(a, m[0], m[1], m[2], m[3], m[4], m[5], m[8]);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  {
    ProfScope ps(st, "window_dkv");
    const int items = a.n_snk + (a.n_kt - a.n_st) * a.n_bh * a.nck;
    const win::Behind b(dim3(items), bwd_threads(2), DkvSmem<D>::bytes, st);
    e = cudaLaunchKernelEx(&b.cfg, window_dkv_kernel<D, win::kWindow, 2>, a, m[0], m[1], m[2], m[3], m[6], m[7], dq_ctas);
  }
  if (e != cudaSuccess) return e;
  const int first = a.ncs > 1 ? 0 : a.n_st, end = a.nck > 1 ? a.n_kt : a.n_st;
  if (first < end) {
    ProfScope ps(st, "window_dkv_sum");
    const win::Behind b(dim3((end - first) * a.n_bh, D / 4), 256, 0, st);
    e = cudaLaunchKernelEx(&b.cfg, window_dkv_sum_kernel<D, win::kWindow>, a, first);
  }
  return e;
}

}  // namespace

WinBwdWs window_bwd_ws(const WinDims& s) {
  BwdArgs a{};
  a.s = s;
  plan(a);
  const size_t rows = align256(static_cast<size_t>(s.B) * s.Hq * a.Nqp * 4 + 512);   // a tile's read may pass the end
  WinBwdWs w{};
  w.status = 0;
  w.gave_up = 256;
  w.nlse = w.gave_up + kDqCtas * 4;
  w.delta = w.nlse + rows;
  w.part = w.delta + rows;
  w.total = w.part + static_cast<size_t>(part_slots(a)) * 2 * 128 * s.d * 4;
  return w;
}

int launch_window_bwd(const WinDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                      const void* dO, const int32_t* len, void* dQ, void* dK, void* dV, char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WinBwdWs w = window_bwd_ws(s);
  BwdArgs a{};
  a.s = s;
  plan(a);
  a.len = len;
  a.lse = lse;
  a.nlse = reinterpret_cast<float*>(ws + w.nlse);
  a.delta = reinterpret_cast<float*>(ws + w.delta);
  a.dQ = static_cast<bf16*>(dQ);
  a.dK = static_cast<bf16*>(dK);
  a.dV = static_cast<bf16*>(dV);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.status = reinterpret_cast<int32_t*>(ws);
  a.gave_up = reinterpret_cast<int32_t*>(ws + w.gave_up);
  a.wait_ns = wait_limit_ns();
  a.stall = test_stall();
  const int64_t hd = static_cast<int64_t>(s.Hq) * s.d, kd = static_cast<int64_t>(s.Hkv) * s.d;
  CUtensorMap m[9];
  if (int e = win::token_map(&m[0], Q, s.B, s.Nq, s.Hq, s.d, s.qs, a.P, a.tok)) return e;
  if (int e = win::token_map(&m[1], dO, s.B, s.Nq, s.Hq, s.d, hd, a.P, a.tok)) return e;
  if (int e = win::token_map(&m[2], K, s.B, s.N, s.Hkv, s.d, s.ks, 1, 128)) return e;
  if (int e = win::token_map(&m[3], V, s.B, s.N, s.Hkv, s.d, s.vs, 1, 128)) return e;
  if (int e = win::token_map(&m[4], K, s.B, s.N, s.Hkv, s.d, s.ks, 1, 32)) return e;
  if (int e = win::token_map(&m[5], V, s.B, s.N, s.Hkv, s.d, s.vs, 1, 32)) return e;
  if (int e = win::token_map(&m[6], dK, s.B, s.N, s.Hkv, s.d, kd, 1, 32)) return e;
  if (int e = win::token_map(&m[7], dV, s.B, s.N, s.Hkv, s.d, kd, 1, 32)) return e;
  if (int e = win::token_map(&m[8], O, s.B, s.Nq, s.Hq, s.d, hd, a.P, a.tok)) return e;
  return s.d == 128 ? bwd_launch<128>(a, m, st) : bwd_launch<64>(a, m, st);
}

}  // namespace pisa
