// Launches of the documents' backward kernels at one head size (doc_bwd_d64.cu, doc_bwd_d128.cu; a file a size, which compile side by side).
//
// The window's backward kernels (window_bwd.cuh) with documents' ends, behind the kernel that lays the rows out. D = dO . O takes O
// as bf16 has it where a row tile sees more than two key tiles: with peaked scores that rounding adds a tenth to the gradients'
// error (0.0024 to 0.0026 of their size, rms), and would take a second pass over the keys to avoid.
// 8192 tokens, 16 heads over 2, d = 128, one document: dQ 268 us, dK and dV 389, their partial sums 18; capped 303 and 529, biased
// 285 and 478, both 393 and 638.
// 35K tokens in 60 documents of 64 to 2048, 16 heads over 4: 256 and 271 (288 with key tiles in the order of their keys: those that
// many tokens see come first).
#pragma once

#include <algorithm>

#include "doc_rows.cuh"
#include "profile.h"
#include "window_bwd.cuh"

namespace pisa {

namespace {

template <int D, int MASK>
int doc_bwd_launch(const BwdArgs& a, const CUtensorMap* m, cudaStream_t st) {
  // capped scores in dQ's kernel: four threads a row (425 -> 346 us for 8192 rows of 16 heads over 2, all causal, 298 since the cap
  // stays in registers; no gain without a cap, nor in dK, dV's kernel, where 96 registers a thread are too few)
  constexpr int NQ = MASK & win::kCap ? 4 : 2;
  static win::Ready dq_ready, dkv_ready;
  if (int e = dq_ready(window_dq_kernel<D, MASK, NQ>, DqSmem<D>::bytes)) return e;
  if (int e = dkv_ready(window_dkv_kernel<D, MASK, 2>, DkvSmem<D>::bytes)) return e;
  const int dq_ctas = std::min({a.n_items, sm_count(), kDqCtas});
  cudaError_t e;
  {
    ProfScope ps(st, "doc_dq");
    const win::Behind b(dim3(dq_ctas), bwd_threads(NQ), DqSmem<D>::bytes, st);
    e = cudaLaunchKernelEx(&b.cfg, window_dq_kernel<D, MASK, NQ>, a, m[0], m[1], m[2], m[3], m[2], m[3], m[6]);
  }
  if (e != cudaSuccess) return e;
  {
    ProfScope ps(st, "doc_dkv");
    const win::Behind b(dim3(a.n_kt * a.n_bh * a.nck), bwd_threads(2), DkvSmem<D>::bytes, st);
    e = cudaLaunchKernelEx(&b.cfg, window_dkv_kernel<D, MASK, 2>, a, m[0], m[1], m[2], m[3], m[4], m[5], dq_ctas);
  }
  if (e != cudaSuccess || a.nck == 1) return e;
  ProfScope ps(st, "doc_dkv_sum");
  const win::Behind b(dim3(a.n_kt * a.n_bh, D / 4), 256, 0, st);
  return cudaLaunchKernelEx(&b.cfg, window_dkv_sum_kernel<D, MASK>, a, 0);
}

template <int D>
int doc_bwd_by_scores(const BwdArgs& a, const CUtensorMap* m, cudaStream_t st) {
  constexpr int C = win::kDocs | win::kCap, B = win::kDocs | win::kBias;
  if (a.docs.cap > 0.f) return a.docs.slopes ? doc_bwd_launch<D, C | B>(a, m, st) : doc_bwd_launch<D, C>(a, m, st);
  return a.docs.slopes ? doc_bwd_launch<D, B>(a, m, st) : doc_bwd_launch<D, win::kDocs>(a, m, st);
}

// The window's backward workspace, then the documents' rows with tiles of `tok` tokens.
size_t rows_at(const DocDims& s) { return (window_bwd_ws(doc_as_window(s)).total + 255) / 256 * 256; }
int row_tile(const DocDims& s) { return 128 / win::packed_heads(s.G); }

template <int D>
int doc_bwd(const DocDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse, const void* dO,
            const DocMask& m, void* dQ, void* dK, void* dV, char* ws, cudaStream_t st) {
  BwdArgs a{};
  a.s = doc_as_window(s);
  const WinBwdWs w = window_bwd_ws(a.s);
  plan(a);
  a.Q = static_cast<const bf16*>(Q);
  a.K = static_cast<const bf16*>(K);
  a.V = static_cast<const bf16*>(V);
  a.dO = static_cast<const bf16*>(dO);
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
  CUtensorMap map[7];
  if (int e = win::token_map(&map[0], Q, 1, s.T, s.Hq, s.d, s.qs, a.P, a.tok)) return e;
  if (int e = win::token_map(&map[1], dO, 1, s.T, s.Hq, s.d, hd, a.P, a.tok)) return e;
  if (int e = win::token_map(&map[2], K, 1, s.T, s.Hkv, s.d, s.ks, 1, 128)) return e;
  if (int e = win::token_map(&map[3], V, 1, s.T, s.Hkv, s.d, s.vs, 1, 128)) return e;
  if (int e = win::token_map(&map[4], dK, 1, s.T, s.Hkv, s.d, kd, 1, 32)) return e;
  if (int e = win::token_map(&map[5], dV, 1, s.T, s.Hkv, s.d, kd, 1, 32)) return e;
  if (int e = win::token_map(&map[6], O, 1, s.T, s.Hq, s.d, hd, a.P, a.tok)) return e;
  if (int e = launch_doc_rows(s, m, a.tok, true, ws + rows_at(s), a.status, &a.docs, st)) return e;
  return doc_bwd_by_scores<D>(a, map, st);
}

}  // namespace
}  // namespace pisa
