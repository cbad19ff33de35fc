// The documents' rows laid out on the device: every token's document and the order of the token tiles (masks.cuh), where the
// forward and backward kernels want them.
#pragma once

#include "device.cuh"
#include "internal.h"
#include "masks.cuh"
#include "paged.h"
#include "profile.h"

namespace pisa {

namespace {

constexpr int kRowThreads = 512, kStarts = 4096, kBuckets = 256;

struct DocRowsArgs {
  win::DocRows d;
  int32_t tile, n_tiles, shift;                // tokens of a tile; 128s of keys (tokens) of a bucket of the orders, as a power of two
  int4* bounds;
  int32_t *order, *key_order, *status;         // key_order: or NULL; status: the workspace's word, cleared
};

// Block 0 sorts the token tiles, block 1 the key tiles (where their order is wanted), the others look tokens up. The starts are
// held in shared memory where they fit.
__global__ void __launch_bounds__(kRowThreads) doc_rows_kernel(const DocRowsArgs a) {
  __shared__ int32_t s_starts[kStarts];
  __shared__ int32_t s_count[kBuckets];
  win::launch_dependents();
  const win::DocRows& d = a.d;
  const bool held = d.n_docs < kStarts;
  if (held)
    for (int k = threadIdx.x; k <= d.n_docs; k += kRowThreads) s_starts[k] = d.starts[k];
  const int sorts = a.key_order ? 2 : 1;
  if (static_cast<int>(blockIdx.x) < sorts)
    for (int k = threadIdx.x; k < kBuckets; k += kRowThreads) s_count[k] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  __syncthreads();
  auto start_of = [&](int m) { return held ? s_starts[m] : d.starts[m]; };
  auto bounds_of = [&](int t) { return d.search(t, start_of); };
  if (static_cast<int>(blockIdx.x) >= sorts) {
    const int t = static_cast<int>((blockIdx.x - sorts) * kRowThreads + threadIdx.x);
    if (t < d.T) a.bounds[t] = bounds_of(t);
    if (t == d.T) a.bounds[t] = make_int4(d.clamped(start_of(0)), d.clamped(start_of(d.n_docs)), 0, 0);
    return;
  }
  const bool keys = blockIdx.x == 1;
  const int tile = keys ? 128 : a.tile, n_tiles = keys ? (d.T + 127) / 128 : a.n_tiles;
  int32_t* order = keys ? a.key_order : a.order;
  auto bucket_of = [&](int k) {                        // what token tile k sees, or key tile k is seen by
    const int t1 = min(d.T, (k + 1) * tile) - 1;
    const int4 p = bounds_of(k * tile), q = bounds_of(t1);
    const int last = keys || t1 >= q.y ? q.y - 1 : max(t1, q.z - 1), first = keys && k * tile >= p.z ? max(p.x, k * tile) : p.x;
    return kBuckets - 1 - min(kBuckets - 1, max(0, (last - first + 128) >> 7) >> a.shift);
  };
  for (int k = threadIdx.x; k < n_tiles; k += kRowThreads) atomicAdd(&s_count[bucket_of(k)], 1);
  __syncthreads();
  if (threadIdx.x < 32) {                              // counts to places
    int before = 0;
    for (int k = threadIdx.x; k < kBuckets; k += 32) {
      const int n = s_count[k];
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (static_cast<int>(threadIdx.x) >= o) sum += x;
      }
      s_count[k] = before + sum - n;
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < n_tiles; k += kRowThreads) order[atomicAdd(&s_count[bucket_of(k)], 1)] = k;
}

inline size_t doc_bounds_bytes(const DocDims& s) { return (static_cast<size_t>(s.T + 1) * 16 + 255) / 256 * 256; }

// Bytes of the rows with token tiles of `tile` tokens; keys: and the key tiles' order.
inline size_t doc_rows_bytes(const DocDims& s, int tile, bool keys) {
  return doc_bounds_bytes(s) + (static_cast<size_t>((s.T + tile - 1) / tile) + (keys ? (s.T + 127) / 128 : 0)) * 4;
}

inline win::DocRows doc_rows_searched(const DocDims& s, const DocMask& m) {
  return {nullptr, nullptr, nullptr, m.slopes, s.cap, s.T, s.n_docs, m.starts, m.prefix};
}

inline int launch_doc_rows(const DocDims& s, const DocMask& m, int tile, bool keys, char* ws, int32_t* status, win::DocRows* out,
                           cudaStream_t st) {
  DocRowsArgs a{};
  a.d = doc_rows_searched(s, m);
  a.tile = tile;
  a.n_tiles = (s.T + tile - 1) / tile;
  while ((s.max_len / 128 + 3) >> a.shift >= kBuckets) ++a.shift;
  a.bounds = reinterpret_cast<int4*>(ws);
  a.order = reinterpret_cast<int32_t*>(ws + doc_bounds_bytes(s));
  a.key_order = keys ? a.order + a.n_tiles : nullptr;
  a.status = status;
  *out = a.d;
  out->bounds = a.bounds;
  out->order = a.order;
  out->key_order = a.key_order;
  ProfScope ps(st, "doc_rows");
  doc_rows_kernel<<<(keys ? 3 : 2) + s.T / kRowThreads, kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// The documents' shape as the window's kernels take it: one sequence, no sinks, a window of the longest document.
inline WinDims doc_as_window(const DocDims& s) {
  WinDims d{};
  d.B = 1;
  d.Nq = d.N = s.T;
  d.Hq = s.Hq;
  d.Hkv = s.Hkv;
  d.d = s.d;
  d.G = s.G;
  d.window = s.max_len;
  d.scale = s.scale;
  d.qs = s.qs;
  d.ks = s.ks;
  d.vs = s.vs;
  return d;
}

}  // namespace
}  // namespace pisa
