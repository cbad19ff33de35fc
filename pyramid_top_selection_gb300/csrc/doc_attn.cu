// Attention over packed documents, forward: the documents' rows, and launches of window_fwd.cuh's kernel.
//
// A token sees one run of keys of its own document, [start, max(t, start + prefix - 1)], and spans neither begin nor end
// before an earlier token's: so a tile of tokens sees one run as well, whether it lies in one document or over several, and the
// window's kernels walk it with other ends (masks.cuh). Where there are many items, a first, small kernel looks every token's
// document up (16 bytes a token), sorts the token tiles by their keys, the most first, and clears the status word; the
// attention's kernel is launched behind it while it runs.
//
// Bound by the window kernel's MMA warp where scores are as they are, by the softmax warps' chain where they are capped
// (masks.cuh). Six prompts of 1500 to 8192 tokens, 16 heads over 2, d = 128: 423 us (1.52 PFLOP/s of what tokens see), biased
// 480-494, capped 680 (945 TFLOP/s), both 722; with scores beyond the polynomial's range (a cap of 10) 831. 35K tokens in 60
// documents of 64 to 2048, 16 heads over 4: 190 us, a fifth of whose tiles' area is not seen; biased 211, capped 290.
#include <algorithm>

#include "doc_rows.cuh"
#include "profile.h"
#include "tmap.h"
#include "window_fwd.cuh"

namespace pisa {

namespace {

template <int D, int MASK>
int doc_fwd_launch(const FwdArgs& a, const CUtensorMap* m, cudaStream_t st) {
  static win::Ready ready;
  // (the softmax warps' larger register share is drawn from what the CTA was launched with: 168 a thread)
  if (int e = ready(window_fwd_kernel<D, false, MASK>, FwdSmem<D>::bytes, 168)) return e;
  ProfScope ps(st, "doc_fwd");
  const win::Behind b(dim3(static_cast<unsigned>(std::min(a.n_items, sm_count()))), kFwdThreads, FwdSmem<D>::bytes, st);
  return cudaLaunchKernelEx(&b.cfg, window_fwd_kernel<D, false, MASK>, a, m[0], m[1], m[2], m[1], m[2], m[3]);
}

template <int D, int SEARCH>
int doc_fwd_by_scores(const FwdArgs& a, const CUtensorMap* m, cudaStream_t st) {
  constexpr int N = win::kDocs | SEARCH, C = N | win::kCap, B = N | win::kBias;
  if (a.docs.cap > 0.f) return a.docs.slopes ? doc_fwd_launch<D, C | B>(a, m, st) : doc_fwd_launch<D, C>(a, m, st);
  return a.docs.slopes ? doc_fwd_launch<D, B>(a, m, st) : doc_fwd_launch<D, N>(a, m, st);
}

// Tokens of a forward item, two row tiles, and the items.
int fwd_tile(const DocDims& s) { return 2 * 128 / win::packed_heads(s.G); }
int64_t fwd_items(const DocDims& s) {                              // < T Hq
  return static_cast<int64_t>((s.T + fwd_tile(s) - 1) / fwd_tile(s)) * s.Hkv * (s.G / win::packed_heads(s.G));
}

// With no more than an item a CTA the kernel that lays the rows out would cost more than their searches (300 tokens of 4
// heads: 25.6 us a call with it, 17.6 without).
bool rows_laid_out(const DocDims& s) { return fwd_items(s) > win::kPlanSms; }

}  // namespace

size_t doc_fwd_ws(const DocDims& s) { return 256 + (rows_laid_out(s) ? doc_rows_bytes(s, fwd_tile(s), false) : 0); }

int launch_doc_fwd(const DocDims& s, const void* Q, const void* K, const void* V, const DocMask& m, void* O, float* lse,
                   char* ws, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  FwdArgs a{};
  a.s = doc_as_window(s);
  a.Q = static_cast<const __nv_bfloat16*>(Q);
  a.K = static_cast<const __nv_bfloat16*>(K);
  a.V = static_cast<const __nv_bfloat16*>(V);
  a.O = static_cast<__nv_bfloat16*>(O);
  a.lse = lse;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.wait_ns = wait_limit_ns();
  a.stall = test_stall();
  a.P = win::packed_heads(s.G);
  a.lp = win::log2_of(a.P);
  a.tok = 128 / a.P;
  a.n_tiles = (s.T + 2 * a.tok - 1) / (2 * a.tok);
  a.n_heads = s.Hkv * (s.G / a.P);
  a.n_items = static_cast<int>(fwd_items(s));
  a.splits = 1;
  CUtensorMap map[4];
  if (int e = win::token_map(&map[0], Q, 1, s.T, s.Hq, s.d, s.qs, a.P, a.tok)) return e;
  if (int e = win::token_map(&map[1], K, 1, s.T, s.Hkv, s.d, s.ks, 1, 128)) return e;
  if (int e = win::token_map(&map[2], V, 1, s.T, s.Hkv, s.d, s.vs, 1, 128)) return e;
  if (int e = win::token_map(&map[3], O, 1, s.T, s.Hq, s.d, static_cast<int64_t>(s.Hq) * s.d, a.P, 32 / a.P)) return e;
  if (!rows_laid_out(s)) {
    a.docs = doc_rows_searched(s, m);
    if (ws) {
      cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
      if (e != cudaSuccess) return e;
    }
    return s.d == 128 ? doc_fwd_by_scores<128, win::kSearch>(a, map, st) : doc_fwd_by_scores<64, win::kSearch>(a, map, st);
  }
  if (int e = launch_doc_rows(s, m, 2 * a.tok, false, ws + 256, a.status, &a.docs, st)) return e;
  return s.d == 128 ? doc_fwd_by_scores<128, 0>(a, map, st) : doc_fwd_by_scores<64, 0>(a, map, st);
}

}  // namespace pisa
