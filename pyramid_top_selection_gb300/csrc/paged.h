// Host-side declarations of the documents' attention and of the paged cache (api.cpp checks the arguments and
// calls these).
#pragma once

#include <cstddef>
#include <cstdint>

#include "window.h"

namespace pisa {

struct DocDims {
  int32_t T, Hq, Hkv, d, G, n_docs, max_len;
  float scale, cap;
  int64_t qs, ks, vs;
};
size_t doc_fwd_ws(const DocDims& s);
size_t doc_bwd_ws(const DocDims& s);

// The device arrays that say what a document's row sees and what its scores become.
struct DocMask {
  const int32_t *starts, *prefix;
  const float* slopes;
};

struct PagedDims {
  int32_t B, Hq, Hkv, d, G, n_pages, page, log_page, max_pages, bits, nq;
  float scale, cap;
};
size_t paged_attn_ws(const PagedDims& s);

struct PagedCache {
  unsigned char *k, *v, *ks, *vs;
  const float *k_amp, *v_amp;
};

// Launchers: return 0 or a cudaError_t value.
int launch_doc_fwd(const DocDims& s, const void* Q, const void* K, const void* V, const DocMask& m, void* O, float* lse,
                   char* ws, void* stream);
int launch_doc_bwd_d64(const DocDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                       const void* dO, const DocMask& m, void* dQ, void* dK, void* dV, char* ws, void* stream);
int launch_doc_bwd_d128(const DocDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                        const void* dO, const DocMask& m, void* dQ, void* dK, void* dV, char* ws, void* stream);
int launch_paged_append(const PagedDims& s, const PagedCache& c, const RopeDims& t, const void* Q, const void* K,
                        const void* V, int64_t vs, const float* inv_freq, const float* wq, const float* wk,
                        const int32_t* table, const int32_t* seq, const int32_t* pos, void* Qr, int32_t* status,
                        void* stream);
int launch_paged_attn(const PagedDims& s, const PagedCache& c, const int32_t* table, const int32_t* len, const void* q,
                      const float* slopes, void* o, float* lse, char* ws, void* stream);

}  // namespace pisa
