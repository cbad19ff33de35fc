// The documents' backward at a head size of 128.
#include "doc_bwd.cuh"
#include "tmap.h"

namespace pisa {

int launch_doc_bwd_d128(const DocDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                       const void* dO, const DocMask& m, void* dQ, void* dK, void* dV, char* ws, void* stream) {
  return doc_bwd<128>(s, Q, K, V, O, lse, dO, m, dQ, dK, dV, ws, static_cast<cudaStream_t>(stream));
}

size_t doc_bwd_ws(const DocDims& s) { return rows_at(s) + doc_rows_bytes(s, row_tile(s), true); }

}  // namespace pisa
