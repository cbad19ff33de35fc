// Host-side declarations of the sliding-window attention and of the query/key norm with
// rotation (api.cpp checks the arguments and calls these).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

namespace pisa {

namespace win {

// The SM count that plans with a host-only size query go by, which have to give the same sizes without a GPU
// (launches ask sm_count()).
constexpr int kPlanSms = 152;

// A kernel's dynamic shared memory, raised once per device (the attribute stays with the device's
// context, and the call costs as much as a launch); `regs` registers a thread must have been compiled.
// `wide_cluster`: clusters of more than 8 CTAs are launched.
class Ready {
 public:
  template <class F>
  int operator()(F* kernel, int bytes, int regs = 0, bool wide_cluster = false) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done_.load(std::memory_order_acquire) & bit) return 0;
    if (regs > 0) {
      cudaFuncAttributes f;
      e = cudaFuncGetAttributes(&f, kernel);
      if (e != cudaSuccess) return e;
      if (f.numRegs < regs) return static_cast<int>(cudaErrorInvalidKernelImage);
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && wide_cluster) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace win

// Plain-old-data view of a window shape, passed to kernels by value. Strides in elements
// between tokens; off = N - Nq is the first query's position.
struct WinDims {
  int32_t B, Nq, N, Hq, Hkv, d, G, off, window, sinks;
  float scale;
  int64_t qs, ks, vs;
};

struct WinBwdWs {
  size_t status, gave_up, nlse, delta, part, total;
};
WinBwdWs window_bwd_ws(const WinDims& s);

struct WinDecodeDims {
  int32_t B, Ncap, Hq, Hkv, d, G, window, sinks;
  float scale;
};

struct RopeDims {
  int32_t B, N, Hq, Hkv, d, rot, interleaved, norm;
  float eps, rot_scale;
  int64_t qs, ks;
};
size_t rope_bwd_ws(const RopeDims& s);

// Launchers: return 0 or a cudaError_t value.
int launch_window_fwd(const WinDims& s, const void* Q, const void* K, const void* V, const int32_t* len, void* O,
                      float* lse, char* ws, void* stream);
int launch_window_bwd(const WinDims& s, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                      const void* dO, const int32_t* len, void* dQ, void* dK, void* dV, char* ws, void* stream);
int launch_window_decode(const WinDecodeDims& s, const int32_t* pos, void* Kc, void* Vc, const void* q,
                         const void* k_new, const void* v_new, void* o, float* lse, int32_t* status, void* stream);
int launch_rope(const RopeDims& s, const void* Q, const void* K, const float* inv_freq, const float* wq,
                const float* wk, const int32_t* pos, void* Qr, void* Kr, void* stream);
int launch_rope_bwd(const RopeDims& s, const void* Q, const void* K, const void* dQr, const void* dKr,
                    const float* inv_freq, const float* wq, const float* wk, const int32_t* pos, void* dQ, void* dK,
                    float* dwq, float* dwk, char* ws, void* stream);

}  // namespace pisa
