// C ABI of the PISA GB300 library: argument checks on the host (before any CUDA call),
// workspace sizing, and dispatch to the kernel launchers.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "internal.h"
#include "window.h"

namespace {

thread_local char g_err[512] = "";

constexpr uint64_t kDefaultWaitNs = 1000000000ull;   // one second
std::atomic<uint64_t> g_wait_ns{kDefaultWaitNs};
std::atomic<int> g_stall{0};

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_ptr(const void* p, const char* name, bool nullable = false) {
  if (!p) return nullable ? PISA_OK : fail(PISA_EINVAL, "%s is NULL", name);
  if (!aligned16(p)) return fail(PISA_EINVAL, "%s is not 16-byte aligned", name);
  return PISA_OK;
}

#define PISA_CHECK(expr)          \
  do {                            \
    const int _rc = (expr);       \
    if (_rc != PISA_OK) return _rc; \
  } while (0)

int check_common(int B, int N, int Hq, int Hkv, int d, int C, int K, int g) {
  if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || d < 1 || C < 1 || K < 1 || g < 1)
    return fail(PISA_EINVAL, "sizes must be positive (B=%d N=%d Hq=%d Hkv=%d d=%d C=%d K=%d g=%d)",
                B, N, Hq, Hkv, d, C, K, g);
  if (Hq % Hkv != 0) return fail(PISA_EINVAL, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
  const int G = Hq / Hkv;
  if (d != 64 && d != 128) return fail(PISA_EUNSUPPORTED, "head dim d=%d (supported: 64, 128)", d);
  if (C != 64) return fail(PISA_EUNSUPPORTED, "leaf block C=%d (supported: 64)", C);
  if (g != 2 && g != 4)
    return fail(PISA_EUNSUPPORTED, "fan-out g=%d (supported: 2, the merge factor, and 4, two levels per step)", g);
  if (K > 32) return fail(PISA_EUNSUPPORTED, "K=%d (supported: 1..32)", K);
  if (g * K > 64) return fail(PISA_EUNSUPPORTED, "g*K=%d candidates (supported: at most 64)", g * K);
  if (G != 1 && G != 2 && G != 4 && G != 8)
    return fail(PISA_EUNSUPPORTED, "GQA group G=%d (supported: 1, 2, 4, 8)", G);
  if (N > (1 << 24)) return fail(PISA_EUNSUPPORTED, "N=%d exceeds 2^24", N);
  const int64_t pairs = static_cast<int64_t>(B) * Hkv * N * g * K;
  if (pairs >= (int64_t(1) << 31))
    return fail(PISA_EUNSUPPORTED, "B*Hkv*N*gK=%lld exceeds 2^31", static_cast<long long>(pairs));
  const int64_t rows = static_cast<int64_t>(B) * N * Hq;   // TMA row coordinates are int32
  if (rows >= (int64_t(1) << 31))
    return fail(PISA_EUNSUPPORTED, "B*N*Hq=%lld exceeds 2^31", static_cast<long long>(rows));
  return PISA_OK;
}

int check_shape(const pisa_shape_t* s) {
  if (!s) return fail(PISA_EINVAL, "shape is NULL");
  PISA_CHECK(check_common(s->B, s->N, s->Hq, s->Hkv, s->d, s->C, s->K, s->g));
  if (s->qtile < 0) return fail(PISA_EINVAL, "qtile=%d is negative", s->qtile);
  if (s->per_head != 0 && s->per_head != 1) return fail(PISA_EINVAL, "per_head=%d (0 or 1)", s->per_head);
  if (s->per_head) {          // the units are the query heads
    const int64_t pairs = static_cast<int64_t>(s->B) * s->Hq * s->N * s->g * s->K;
    if (pairs >= (int64_t(1) << 31))
      return fail(PISA_EUNSUPPORTED, "B*Hq*N*gK=%lld exceeds 2^31 (per-head selection)", static_cast<long long>(pairs));
  }
  if (!(s->scale >= 0.f) || std::isinf(s->scale)) return fail(PISA_EINVAL, "scale must be finite and >= 0");
  return PISA_OK;
}

pisa::Dims dims_of(const pisa_shape_t* s) {
  pisa::Dims d{};
  d.B = s->B; d.N = s->N; d.Hq = s->Hq; d.Hkv = s->Hkv; d.d = s->d; d.C = s->C; d.K = s->K;
  d.G = s->Hq / s->Hkv;
  d.n0 = (s->N + s->C - 1) / s->C;
  d.scale = s->scale > 0.f ? s->scale : 1.0f / std::sqrt(static_cast<float>(s->d));
  d.Hkv_r = s->Hkv;
  d.kvr = 1;
  d.g = s->g;
  if (s->per_head) {          // every query head a selection unit of its own
    d.kvr = d.G;
    d.Hkv = s->Hq;
    d.G = 1;
  }
  return d;
}

// The real (per KV head) view of a shape, for the pyramid build: the pyramid always belongs to
// the KV heads.
pisa::Dims kv_dims_of(const pisa_shape_t* s) {
  pisa_shape_t r = *s;
  r.per_head = 0;
  return dims_of(&r);
}

pisa::Dims dims_of(const pisa_decode_shape_t* s) {
  pisa::Dims d{};
  d.B = s->B; d.N = s->Ncap; d.Hq = s->Hq; d.Hkv = s->Hkv; d.d = s->d; d.C = s->C; d.K = s->K;
  d.G = s->Hq / s->Hkv;
  d.n0 = (s->Ncap + s->C - 1) / s->C;
  d.scale = s->scale > 0.f ? s->scale : 1.0f / std::sqrt(static_cast<float>(s->d));
  d.Hkv_r = s->Hkv;
  d.kvr = 1;
  d.g = s->g;
  return d;
}

int cuda_rc(int err, const char* what) {
  if (err == 0) return PISA_OK;
  return fail(PISA_ECUDA, "%s: CUDA error %d (%s)", what, err, pisa::cuda_error_string(err));
}

int layout_out(const pisa::Geo& g, int32_t* n_levels, int64_t* level_offset, int64_t* nodes) {
  if (n_levels) *n_levels = g.n_levels;
  if (level_offset)
    for (int l = 0; l < g.n_levels; ++l) level_offset[l] = g.off[l];
  if (nodes) *nodes = g.nodes;
  return PISA_OK;
}

size_t ws_bytes_for(const pisa::Dims& d, const pisa::Geo& g, int op) {
  switch (op) {
    case PISA_OP_SELECT: return pisa::select_ws(d, g).total_head;
    case PISA_OP_SELECT_MEAN: return pisa::select_ws(d, g).mean_end;
    case PISA_OP_SELECT_MEANVAR: return pisa::meanvar_ws(d, g);
    case PISA_OP_SELECT_FLAT: return pisa::flat_ws(d, g);
    case PISA_OP_ATTN_FWD: return pisa::attn_fwd_ws(d).total;
    case PISA_OP_ATTN_BWD: return pisa::attn_bwd_ws(d).total;
    default: return 0;
  }
}

int check_ws_bytes(size_t need, const void* ws, size_t ws_bytes) {
  if (ws_bytes < need) return fail(PISA_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
  if (need > 0 && !ws) return fail(PISA_EWORKSPACE, "workspace is NULL");
  if (ws && !aligned16(ws)) return fail(PISA_EINVAL, "workspace is not 16-byte aligned");
  return PISA_OK;
}

int check_ws(const pisa::Dims& d, const pisa::Geo& g, int op, const void* ws, size_t ws_bytes) {
  return check_ws_bytes(ws_bytes_for(d, g, op), ws, ws_bytes);
}

// ---- sliding-window attention, query/key norm with rotation

int check_heads(int Hq, int Hkv, int d) {
  if (Hq % Hkv != 0) return fail(PISA_EINVAL, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
  if (d != 64 && d != 128) return fail(PISA_EUNSUPPORTED, "head dim d=%d (supported: 64, 128)", d);
  return PISA_OK;
}

int check_scale(float scale, const char* name) {
  if (!(scale >= 0.f) || std::isinf(scale)) return fail(PISA_EINVAL, "%s must be finite and >= 0", name);
  return PISA_OK;
}

// Token stride in elements: 0 means contiguous.
int check_stride(int32_t stride, int H, int d, const char* name, int64_t* out) {
  const int64_t row = static_cast<int64_t>(H) * d;
  if (stride != 0 && (stride < row || stride % 8 != 0))
    return fail(PISA_EINVAL, "%s=%d must be 0 or a multiple of 8 of at least H*d=%lld", name, stride,
                static_cast<long long>(row));
  *out = stride ? stride : row;
  return PISA_OK;
}

// A buffer's bytes; `tokens` rows of `row` elements, `stride` elements apart.
struct Span {
  const char* name;
  uintptr_t begin, end;
  Span(const char* n, const void* p, int64_t tokens, int64_t stride, int64_t row, int bytes = 2)
      : name(n), begin(reinterpret_cast<uintptr_t>(p)),
        end(p ? begin + static_cast<uintptr_t>(((tokens - 1) * stride + row) * bytes) : begin) {}
};

// One value, or `n` of `bytes` bytes in a row.
Span flat(const char* name, const void* p, int64_t n, int bytes) { return Span(name, p, 1, 0, n, bytes); }

// What is written shares no bytes with what is read, nor with anything else that is written; of the first
// `in_place` buffers, the k-th written may be the k-th read.
template <int NIN, int NOUT>
int check_apart(const Span (&in)[NIN], const Span (&out)[NOUT], int in_place = 0) {
  auto meet = [](const Span& a, const Span& b) { return a.begin < b.end && b.begin < a.end; };
  for (int o = 0; o < NOUT; ++o) {
    for (int i = 0; i < NIN; ++i) {
      if (i == o && i < in_place && in[i].begin == out[o].begin) continue;
      if (meet(out[o], in[i])) return fail(PISA_EINVAL, "%s overlaps %s", out[o].name, in[i].name);
    }
    for (int k = 0; k < o; ++k)
      if (meet(out[o], out[k])) return fail(PISA_EINVAL, "%s overlaps %s", out[o].name, out[k].name);
  }
  return PISA_OK;
}

float scale_or_default(float scale, int d) { return scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(d)); }

int window_dims(const pisa_window_shape_t* s, pisa::WinDims* o) {
  if (!s) return fail(PISA_EINVAL, "shape is NULL");
  if (s->B < 1 || s->Nq < 1 || s->N < 1 || s->Hq < 1 || s->Hkv < 1 || s->d < 1 || s->window < 1)
    return fail(PISA_EINVAL, "sizes must be positive (B=%d Nq=%d N=%d Hq=%d Hkv=%d d=%d window=%d)", s->B, s->Nq,
                s->N, s->Hq, s->Hkv, s->d, s->window);
  if (s->sinks < 0) return fail(PISA_EINVAL, "sinks=%d is negative", s->sinks);
  if (s->Nq > s->N) return fail(PISA_EINVAL, "Nq=%d exceeds N=%d", s->Nq, s->N);
  PISA_CHECK(check_heads(s->Hq, s->Hkv, s->d));
  if (s->Hq / s->Hkv > 64) return fail(PISA_EUNSUPPORTED, "GQA group G=%d (supported: at most 64)", s->Hq / s->Hkv);
  if (s->N > (1 << 24)) return fail(PISA_EUNSUPPORTED, "N=%d exceeds 2^24", s->N);
  const int64_t bn = static_cast<int64_t>(s->B) * s->N;
  if (bn >= (int64_t(1) << 31) || bn * s->Hq >= (int64_t(1) << 31))
    return fail(PISA_EUNSUPPORTED, "B*N*Hq=%lld exceeds 2^31", static_cast<long long>(bn * s->Hq));
  PISA_CHECK(check_scale(s->scale, "scale"));
  pisa::WinDims d{};
  PISA_CHECK(check_stride(s->q_stride, s->Hq, s->d, "q_stride", &d.qs));
  PISA_CHECK(check_stride(s->k_stride, s->Hkv, s->d, "k_stride", &d.ks));
  PISA_CHECK(check_stride(s->v_stride, s->Hkv, s->d, "v_stride", &d.vs));
  const int64_t strides[] = {d.qs, d.ks, d.vs};      // TMA: less than 2^40 bytes between batches
  for (const int64_t st : strides)
    if (st * s->N >= (int64_t(1) << 39)) return fail(PISA_EUNSUPPORTED, "token stride %lld at N=%d", static_cast<long long>(st), s->N);
  d.B = s->B; d.Nq = s->Nq; d.N = s->N; d.Hq = s->Hq; d.Hkv = s->Hkv; d.d = s->d;
  d.G = s->Hq / s->Hkv;
  d.off = s->N - s->Nq;
  // the same keys, and no sum of positions overflows
  d.window = s->window < s->N ? s->window : s->N;
  d.sinks = s->sinks < s->N ? s->sinks : s->N;
  if (d.window + d.sinks >= s->N) {                   // no key lies between sinks and window: full causal attention
    d.window = s->N;
    d.sinks = 0;
  }
  d.scale = scale_or_default(s->scale, s->d);
  *o = d;
  return PISA_OK;
}

size_t window_ws_bytes(const pisa::WinDims& d, int op) {
  return op == PISA_WINDOW_FWD ? 256 : pisa::window_bwd_ws(d).total;
}

int window_decode_dims(const pisa_window_decode_shape_t* s, pisa::WinDecodeDims* o) {
  if (!s) return fail(PISA_EINVAL, "shape is NULL");
  if (s->B < 1 || s->Ncap < 1 || s->Hq < 1 || s->Hkv < 1 || s->d < 1 || s->window < 1)
    return fail(PISA_EINVAL, "sizes must be positive (B=%d Ncap=%d Hq=%d Hkv=%d d=%d window=%d)", s->B, s->Ncap,
                s->Hq, s->Hkv, s->d, s->window);
  if (s->sinks < 0) return fail(PISA_EINVAL, "sinks=%d is negative", s->sinks);
  if (s->Ncap <= s->sinks) return fail(PISA_EINVAL, "Ncap=%d must exceed sinks=%d", s->Ncap, s->sinks);
  PISA_CHECK(check_heads(s->Hq, s->Hkv, s->d));
  if (s->Hq / s->Hkv > 64) return fail(PISA_EUNSUPPORTED, "GQA group G=%d (supported: at most 64)", s->Hq / s->Hkv);
  if (s->Ncap > (1 << 24)) return fail(PISA_EUNSUPPORTED, "Ncap=%d exceeds 2^24", s->Ncap);
  if (s->B > 65535 || s->Hq > 65535) return fail(PISA_EUNSUPPORTED, "B=%d or Hq=%d exceeds 65535", s->B, s->Hq);
  PISA_CHECK(check_scale(s->scale, "scale"));
  pisa::WinDecodeDims d{};
  d.B = s->B; d.Ncap = s->Ncap; d.Hq = s->Hq; d.Hkv = s->Hkv; d.d = s->d;
  d.G = s->Hq / s->Hkv;
  d.window = s->window;
  d.sinks = s->sinks;
  d.scale = scale_or_default(s->scale, s->d);
  *o = d;
  return PISA_OK;
}

int rope_dims(const pisa_rope_shape_t* s, pisa::RopeDims* o) {
  if (!s) return fail(PISA_EINVAL, "shape is NULL");
  if (s->B < 1 || s->N < 1 || s->Hq < 1 || s->Hkv < 1 || s->d < 1)
    return fail(PISA_EINVAL, "sizes must be positive (B=%d N=%d Hq=%d Hkv=%d d=%d)", s->B, s->N, s->Hq, s->Hkv, s->d);
  if (s->d != 64 && s->d != 128) return fail(PISA_EUNSUPPORTED, "head dim d=%d (supported: 64, 128)", s->d);
  if (s->rot < 0 || s->rot > s->d) return fail(PISA_EINVAL, "rot=%d is outside [0, d=%d]", s->rot, s->d);
  if (s->rot % 16 != 0) return fail(PISA_EUNSUPPORTED, "rot=%d (supported: multiples of 16)", s->rot);
  if ((s->interleaved != 0 && s->interleaved != 1) || (s->norm != 0 && s->norm != 1))
    return fail(PISA_EINVAL, "interleaved=%d and norm=%d must be 0 or 1", s->interleaved, s->norm);
  PISA_CHECK(check_scale(s->eps, "eps"));
  PISA_CHECK(check_scale(s->rot_scale, "rot_scale"));
  const int64_t bn = static_cast<int64_t>(s->B) * s->N, H = static_cast<int64_t>(s->Hq) + s->Hkv;
  if (bn >= (int64_t(1) << 31) || H >= (int64_t(1) << 31) || bn * H >= (int64_t(1) << 31))
    return fail(PISA_EUNSUPPORTED, "B*N*(Hq+Hkv) exceeds 2^31");
  pisa::RopeDims d{};
  PISA_CHECK(check_stride(s->q_stride, s->Hq, s->d, "q_stride", &d.qs));
  PISA_CHECK(check_stride(s->k_stride, s->Hkv, s->d, "k_stride", &d.ks));
  d.B = s->B; d.N = s->N; d.Hq = s->Hq; d.Hkv = s->Hkv; d.d = s->d; d.rot = s->rot;
  d.interleaved = s->interleaved;
  d.norm = s->norm;
  d.eps = s->eps;
  d.rot_scale = s->rot_scale > 0.f ? s->rot_scale : 1.f;
  *o = d;
  return PISA_OK;
}

}  // namespace

namespace pisa {
uint64_t wait_limit_ns() { return g_wait_ns.load(std::memory_order_relaxed); }
int test_stall() { return g_stall.load(std::memory_order_relaxed); }
}  // namespace pisa

extern "C" {

int pisa_version(void) { return PISA_VERSION; }

const char* pisa_last_error(void) { return g_err; }

int pisa_set_wait_limit(uint64_t limit_ns) {
  g_wait_ns.store(limit_ns == 0 ? kDefaultWaitNs : limit_ns, std::memory_order_relaxed);
  return PISA_OK;
}

int pisa_test_stall(int on) {
  g_stall.store(on ? 1 : 0, std::memory_order_relaxed);
  return PISA_OK;
}

int pisa_pyramid_layout(const pisa_shape_t* shape, int32_t* n_levels, int64_t* level_offset,
                        int64_t* nodes_per_head) {
  PISA_CHECK(check_shape(shape));
  return layout_out(pisa::make_geo(shape->N, shape->C), n_levels, level_offset, nodes_per_head);
}

int pisa_workspace_size(const pisa_shape_t* shape, int op, size_t* bytes) {
  PISA_CHECK(check_shape(shape));
  if (!bytes) return fail(PISA_EINVAL, "bytes is NULL");
  if (op < PISA_OP_SELECT || op > PISA_OP_SELECT_MEANVAR) return fail(PISA_EINVAL, "unknown op %d", op);
  *bytes = ws_bytes_for(dims_of(shape), pisa::make_geo(shape->N, shape->C), op);
  return PISA_OK;
}

int pisa_build_pyramid(const pisa_shape_t* shape, const void* K, float* pyr_sum, void* stream) {
  PISA_CHECK(check_shape(shape));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(pyr_sum, "pyr_sum"));
  const pisa::Dims d = kv_dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  return cuda_rc(pisa::launch_build_pyramid(d, g, K, nullptr, d.N, pyr_sum, stream), "pisa_build_pyramid");
}

int pisa_select(const pisa_shape_t* shape, const void* Q, const void* K, const float* pyr_sum,
                int32_t* idx, float* score, float* head_lse, void* ws, size_t ws_bytes, void* stream) {
  PISA_CHECK(check_shape(shape));
  PISA_CHECK(check_ptr(Q, "Q"));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(pyr_sum, "pyr_sum"));
  PISA_CHECK(check_ptr(idx, "idx"));
  PISA_CHECK(check_ptr(score, "score", true));
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  PISA_CHECK(check_ptr(head_lse, "head_lse", true));
  PISA_CHECK(check_ws(d, g, PISA_OP_SELECT, ws, ws_bytes));
  return cuda_rc(pisa::launch_select(d, g, Q, K, pyr_sum, idx, score, head_lse, static_cast<char*>(ws), stream),
                 "pisa_select");
}

int pisa_select_noalloc(const pisa_shape_t* shape, const void* Q, const void* K,
                        const float* pyr_sum, int32_t* idx, float* score, void* stream) {
  PISA_CHECK(check_shape(shape));
  PISA_CHECK(check_ptr(Q, "Q"));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(pyr_sum, "pyr_sum"));
  PISA_CHECK(check_ptr(idx, "idx"));
  PISA_CHECK(check_ptr(score, "score", true));
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  const size_t need = pisa::select_ws(d, g, false).total;
  if (need > pisa::noalloc_scratch_bytes())
    return fail(PISA_EUNSUPPORTED,
                "pisa_select_noalloc: this shape needs %zu bytes of scratch, more than the fixed %zu; "
                "use pisa_select with a caller workspace", need, pisa::noalloc_scratch_bytes());
  void* ws = nullptr;
  PISA_CHECK(cuda_rc(pisa::noalloc_scratch(&ws), "pisa_select_noalloc scratch set-up"));
  return cuda_rc(pisa::launch_select(d, g, Q, K, pyr_sum, idx, score, nullptr, static_cast<char*>(ws), stream, false),
                 "pisa_select_noalloc");
}

int pisa_select_flat(const pisa_shape_t* shape, const void* Q, const void* K,
                     const float* pyr_sum, int32_t* idx, float* score, void* ws,
                     size_t ws_bytes, void* stream) {
  PISA_CHECK(check_shape(shape));
  PISA_CHECK(check_ptr(Q, "Q"));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(pyr_sum, "pyr_sum"));
  PISA_CHECK(check_ptr(idx, "idx"));
  PISA_CHECK(check_ptr(score, "score", true));
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  PISA_CHECK(check_ws(d, g, PISA_OP_SELECT_FLAT, ws, ws_bytes));
  return cuda_rc(pisa::launch_select_flat(d, g, Q, K, pyr_sum, idx, score, static_cast<char*>(ws), stream),
                 "pisa_select_flat");
}

int pisa_select_mean(const pisa_shape_t* shape, const void* Q, const void* K,
                     const float* pyr_sum, int32_t* idx, float* score, void* ws,
                     size_t ws_bytes, void* stream) {
  PISA_CHECK(check_shape(shape));
  PISA_CHECK(check_ptr(Q, "Q"));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(pyr_sum, "pyr_sum"));
  PISA_CHECK(check_ptr(idx, "idx"));
  PISA_CHECK(check_ptr(score, "score", true));
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  if (shape->g != 2) return fail(PISA_EUNSUPPORTED, "pisa_select_mean: fan-out g=%d (supported: 2)", shape->g);
  PISA_CHECK(check_ws(d, g, PISA_OP_SELECT_MEAN, ws, ws_bytes));
  return cuda_rc(pisa::launch_select_mean(d, g, Q, K, pyr_sum, idx, score, static_cast<char*>(ws), stream),
                 "pisa_select_mean");
}

int pisa_select_meanvar(const pisa_shape_t* shape, const void* Q, const void* K,
                        const float* pyr_sum, int32_t* idx, float* score, void* ws,
                        size_t ws_bytes, void* stream) {
  PISA_CHECK(check_shape(shape));
  PISA_CHECK(check_ptr(Q, "Q"));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(pyr_sum, "pyr_sum"));
  PISA_CHECK(check_ptr(idx, "idx"));
  PISA_CHECK(check_ptr(score, "score", true));
  if (shape->g != 2) return fail(PISA_EUNSUPPORTED, "pisa_select_meanvar: fan-out g=%d (supported: 2)", shape->g);
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  PISA_CHECK(check_ws(d, g, PISA_OP_SELECT_MEANVAR, ws, ws_bytes));
  return cuda_rc(pisa::launch_select_meanvar(d, g, Q, K, pyr_sum, idx, score, static_cast<char*>(ws), stream),
                 "pisa_select_meanvar");
}

int pisa_sparse_attn_fwd(const pisa_shape_t* shape, const void* Q, const void* K, const void* V,
                         const int32_t* idx, const float* head_lse, void* O, float* lse, void* ws,
                         size_t ws_bytes, void* stream) {
  PISA_CHECK(check_shape(shape));
  PISA_CHECK(check_ptr(Q, "Q"));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(V, "V"));
  PISA_CHECK(check_ptr(idx, "idx"));
  PISA_CHECK(check_ptr(O, "O"));
  PISA_CHECK(check_ptr(lse, "lse"));
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  PISA_CHECK(check_ptr(head_lse, "head_lse", true));
  PISA_CHECK(check_ws(d, g, PISA_OP_ATTN_FWD, ws, ws_bytes));
  return cuda_rc(pisa::launch_attn_fwd(d, Q, K, V, idx, head_lse, O, lse, static_cast<char*>(ws), stream),
                 "pisa_sparse_attn_fwd");
}

int pisa_sparse_attn_bwd(const pisa_shape_t* shape, const void* Q, const void* K, const void* V,
                         const void* O, const float* lse, const void* dO, const int32_t* idx,
                         void* dQ, void* dK, void* dV, void* ws, size_t ws_bytes, void* stream) {
  PISA_CHECK(check_shape(shape));
  const void* in[] = {Q, K, V, O, lse, dO, idx, dQ, dK, dV};
  const char* names[] = {"Q", "K", "V", "O", "lse", "dO", "idx", "dQ", "dK", "dV"};
  for (int k = 0; k < 10; ++k) PISA_CHECK(check_ptr(in[k], names[k]));
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  PISA_CHECK(check_ws(d, g, PISA_OP_ATTN_BWD, ws, ws_bytes));
  return cuda_rc(pisa::launch_attn_bwd(d, Q, K, V, O, lse, dO, idx, dQ, dK, dV, static_cast<char*>(ws), stream),
                 "pisa_sparse_attn_bwd");
}

int pisa_decode_pyramid_layout(const pisa_decode_shape_t* shape, int32_t* n_levels,
                               int64_t* level_offset, int64_t* nodes_per_head) {
  if (!shape) return fail(PISA_EINVAL, "shape is NULL");
  PISA_CHECK(check_common(shape->B, shape->Ncap, shape->Hq, shape->Hkv, shape->d, shape->C, shape->K, shape->g));
  if (shape->g != 2) return fail(PISA_EUNSUPPORTED, "decode: fan-out g=%d (supported: 2)", shape->g);
  return layout_out(pisa::make_geo(shape->Ncap, shape->C), n_levels, level_offset, nodes_per_head);
}

int pisa_decode_build_pyramid(const pisa_decode_shape_t* shape, const void* Kcache,
                              const int32_t* len, float* pyr_sum, void* stream) {
  if (!shape) return fail(PISA_EINVAL, "shape is NULL");
  PISA_CHECK(check_common(shape->B, shape->Ncap, shape->Hq, shape->Hkv, shape->d, shape->C, shape->K, shape->g));
  if (shape->g != 2) return fail(PISA_EUNSUPPORTED, "decode: fan-out g=%d (supported: 2)", shape->g);
  PISA_CHECK(check_ptr(Kcache, "Kcache"));
  PISA_CHECK(check_ptr(len, "len"));
  PISA_CHECK(check_ptr(pyr_sum, "pyr_sum"));
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  return cuda_rc(pisa::launch_build_pyramid(d, g, Kcache, len, d.N, pyr_sum, stream),
                 "pisa_decode_build_pyramid");
}

int pisa_decode_step(const pisa_decode_shape_t* shape, const int32_t* pos, void* Kcache,
                     void* Vcache, float* pyr_sum, const void* q, const void* k_new,
                     const void* v_new, void* o, int32_t* idx, float* score, int32_t* status,
                     void* stream) {
  if (!shape) return fail(PISA_EINVAL, "shape is NULL");
  PISA_CHECK(check_common(shape->B, shape->Ncap, shape->Hq, shape->Hkv, shape->d, shape->C, shape->K, shape->g));
  if (shape->g != 2) return fail(PISA_EUNSUPPORTED, "decode: fan-out g=%d (supported: 2)", shape->g);
  if (!(shape->scale >= 0.f) || std::isinf(shape->scale)) return fail(PISA_EINVAL, "scale must be finite and >= 0");
  const void* in[] = {pos, Kcache, Vcache, pyr_sum, q, k_new, v_new, o, idx, status};
  const char* names[] = {"pos", "Kcache", "Vcache", "pyr_sum", "q", "k_new", "v_new", "o", "idx", "status"};
  for (int k = 0; k < 10; ++k) PISA_CHECK(check_ptr(in[k], names[k]));
  PISA_CHECK(check_ptr(score, "score", true));
  const pisa::Dims d = dims_of(shape);
  const pisa::Geo g = pisa::make_geo(d.N, d.C);
  return cuda_rc(pisa::launch_decode_step(d, shape->Ncap, g, pos, Kcache, Vcache, pyr_sum, q, k_new,
                                          v_new, o, idx, score, status, stream),
                 "pisa_decode_step");
}

int pisa_window_workspace_size(const pisa_window_shape_t* shape, int op, size_t* bytes) {
  pisa::WinDims d;
  PISA_CHECK(window_dims(shape, &d));
  if (!bytes) return fail(PISA_EINVAL, "bytes is NULL");
  if (op != PISA_WINDOW_FWD && op != PISA_WINDOW_BWD) return fail(PISA_EINVAL, "unknown op %d", op);
  *bytes = window_ws_bytes(d, op);
  return PISA_OK;
}

int pisa_window_attn_fwd(const pisa_window_shape_t* shape, const void* Q, const void* K, const void* V,
                         const int32_t* len, void* O, float* lse, void* ws, size_t ws_bytes, void* stream) {
  pisa::WinDims d;
  PISA_CHECK(window_dims(shape, &d));
  PISA_CHECK(check_ptr(Q, "Q"));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(V, "V"));
  PISA_CHECK(check_ptr(len, "len", true));
  PISA_CHECK(check_ptr(O, "O"));
  PISA_CHECK(check_ptr(lse, "lse"));
  if (ws || ws_bytes) PISA_CHECK(check_ws_bytes(window_ws_bytes(d, PISA_WINDOW_FWD), ws, ws_bytes));
  const int64_t tq = static_cast<int64_t>(d.B) * d.Nq, tk = static_cast<int64_t>(d.B) * d.N;
  const int64_t q = static_cast<int64_t>(d.Hq) * d.d, kv = static_cast<int64_t>(d.Hkv) * d.d;
  const Span in[] = {{"Q", Q, tq, d.qs, q}, {"K", K, tk, d.ks, kv}, {"V", V, tk, d.vs, kv}, flat("len", len, d.B, 4)};
  const Span out[] = {{"O", O, tq, q, q}, {"lse", lse, tq, d.Hq, d.Hq, 4},
                      flat("workspace", ws, static_cast<int64_t>(window_ws_bytes(d, PISA_WINDOW_FWD)), 1)};
  PISA_CHECK(check_apart(in, out));
  return cuda_rc(pisa::launch_window_fwd(d, Q, K, V, len, O, lse, static_cast<char*>(ws), stream),
                 "pisa_window_attn_fwd");
}

int pisa_window_attn_bwd(const pisa_window_shape_t* shape, const void* Q, const void* K, const void* V,
                         const void* O, const float* lse, const void* dO, const int32_t* len, void* dQ,
                         void* dK, void* dV, void* ws, size_t ws_bytes, void* stream) {
  pisa::WinDims d;
  PISA_CHECK(window_dims(shape, &d));
  const void* in[] = {Q, K, V, O, lse, dO, dQ, dK, dV};
  const char* names[] = {"Q", "K", "V", "O", "lse", "dO", "dQ", "dK", "dV"};
  for (int k = 0; k < 9; ++k) PISA_CHECK(check_ptr(in[k], names[k]));
  PISA_CHECK(check_ptr(len, "len", true));
  PISA_CHECK(check_ws_bytes(window_ws_bytes(d, PISA_WINDOW_BWD), ws, ws_bytes));
  const int64_t tq = static_cast<int64_t>(d.B) * d.Nq, tk = static_cast<int64_t>(d.B) * d.N;
  const int64_t q = static_cast<int64_t>(d.Hq) * d.d, kv = static_cast<int64_t>(d.Hkv) * d.d;
  const Span spans[] = {{"Q", Q, tq, d.qs, q}, {"K", K, tk, d.ks, kv}, {"V", V, tk, d.vs, kv}, {"O", O, tq, q, q},
                        {"dO", dO, tq, q, q}, {"lse", lse, tq, d.Hq, d.Hq, 4}, flat("len", len, d.B, 4)};
  const Span out[] = {{"dQ", dQ, tq, q, q}, {"dK", dK, tk, kv, kv}, {"dV", dV, tk, kv, kv},
                      flat("workspace", ws, static_cast<int64_t>(window_ws_bytes(d, PISA_WINDOW_BWD)), 1)};
  PISA_CHECK(check_apart(spans, out));
  return cuda_rc(pisa::launch_window_bwd(d, Q, K, V, O, lse, dO, len, dQ, dK, dV, static_cast<char*>(ws), stream),
                 "pisa_window_attn_bwd");
}

int pisa_window_decode_step(const pisa_window_decode_shape_t* shape, const int32_t* pos, void* Kcache,
                            void* Vcache, const void* q, const void* k_new, const void* v_new, void* o,
                            float* lse, int32_t* status, void* stream) {
  pisa::WinDecodeDims d;
  PISA_CHECK(window_decode_dims(shape, &d));
  const void* in[] = {pos, Kcache, Vcache, q, k_new, v_new, o, status};
  const char* names[] = {"pos", "Kcache", "Vcache", "q", "k_new", "v_new", "o", "status"};
  for (int k = 0; k < 8; ++k) PISA_CHECK(check_ptr(in[k], names[k]));
  PISA_CHECK(check_ptr(lse, "lse", true));
  const int64_t qn = static_cast<int64_t>(d.B) * d.Hq, kn = static_cast<int64_t>(d.B) * d.Hkv * d.d;
  const Span read[] = {flat("q", q, qn * d.d, 2), flat("k_new", k_new, kn, 2), flat("v_new", v_new, kn, 2), flat("pos", pos, d.B, 4)};
  const Span out[] = {flat("o", o, qn * d.d, 2), flat("lse", lse, qn, 4), flat("status", status, 1, 4),
                      flat("Kcache", Kcache, kn * d.Ncap, 2), flat("Vcache", Vcache, kn * d.Ncap, 2)};
  PISA_CHECK(check_apart(read, out, 1));
  return cuda_rc(pisa::launch_window_decode(d, pos, Kcache, Vcache, q, k_new, v_new, o, lse, status, stream),
                 "pisa_window_decode_step");
}

int pisa_qk_norm_rope(const pisa_rope_shape_t* shape, const void* Q, const void* K, const float* inv_freq,
                      const float* q_weight, const float* k_weight, const int32_t* pos, void* Qr, void* Kr,
                      void* stream) {
  pisa::RopeDims d;
  PISA_CHECK(rope_dims(shape, &d));
  PISA_CHECK(check_ptr(Q, "Q"));
  PISA_CHECK(check_ptr(K, "K"));
  PISA_CHECK(check_ptr(inv_freq, "inv_freq", d.rot == 0));
  PISA_CHECK(check_ptr(q_weight, "q_weight", true));
  PISA_CHECK(check_ptr(k_weight, "k_weight", true));
  PISA_CHECK(check_ptr(pos, "pos", true));
  PISA_CHECK(check_ptr(Qr, "Qr"));
  PISA_CHECK(check_ptr(Kr, "Kr"));
  if ((Qr == Q && d.qs != static_cast<int64_t>(d.Hq) * d.d) || (Kr == K && d.ks != static_cast<int64_t>(d.Hkv) * d.d))
    return fail(PISA_EINVAL, "in place needs a contiguous Q and K");
  const int64_t t = static_cast<int64_t>(d.B) * d.N, q = static_cast<int64_t>(d.Hq) * d.d, k = static_cast<int64_t>(d.Hkv) * d.d;
  const Span in[] = {{"Q", Q, t, d.qs, q}, {"K", K, t, d.ks, k}, flat("inv_freq", inv_freq, d.rot / 2, 4),
                     flat("q_weight", q_weight, d.d, 4), flat("k_weight", k_weight, d.d, 4), flat("pos", pos, t, 4)};
  const Span out[] = {{"Qr", Qr, t, q, q}, {"Kr", Kr, t, k, k}};
  PISA_CHECK(check_apart(in, out, 2));
  return cuda_rc(pisa::launch_rope(d, Q, K, inv_freq, q_weight, k_weight, pos, Qr, Kr, stream), "pisa_qk_norm_rope");
}

int pisa_qk_norm_rope_workspace_size(const pisa_rope_shape_t* shape, size_t* bytes) {
  pisa::RopeDims d;
  PISA_CHECK(rope_dims(shape, &d));
  if (!bytes) return fail(PISA_EINVAL, "bytes is NULL");
  *bytes = pisa::rope_bwd_ws(d);
  return PISA_OK;
}

int pisa_qk_norm_rope_bwd(const pisa_rope_shape_t* shape, const void* Q, const void* K, const void* dQr,
                          const void* dKr, const float* inv_freq, const float* q_weight,
                          const float* k_weight, const int32_t* pos, void* dQ, void* dK, float* dq_weight,
                          float* dk_weight, void* ws, size_t ws_bytes, void* stream) {
  pisa::RopeDims d;
  PISA_CHECK(rope_dims(shape, &d));
  const void* in[] = {Q, K, dQr, dKr, dQ, dK};
  const char* names[] = {"Q", "K", "dQr", "dKr", "dQ", "dK"};
  for (int k = 0; k < 6; ++k) PISA_CHECK(check_ptr(in[k], names[k]));
  PISA_CHECK(check_ptr(inv_freq, "inv_freq", d.rot == 0));
  const void* opt[] = {q_weight, k_weight, pos, dq_weight, dk_weight};
  const char* opt_names[] = {"q_weight", "k_weight", "pos", "dq_weight", "dk_weight"};
  for (int k = 0; k < 5; ++k) PISA_CHECK(check_ptr(opt[k], opt_names[k], true));
  if (!d.norm && (dq_weight || dk_weight)) return fail(PISA_EINVAL, "norm=0 has no weight gradients");
  if (dQ == Q || dK == K) return fail(PISA_EINVAL, "dQ and dK must not be Q and K");
  PISA_CHECK(check_ws_bytes(pisa::rope_bwd_ws(d), ws, ws_bytes));
  const int64_t t = static_cast<int64_t>(d.B) * d.N, q = static_cast<int64_t>(d.Hq) * d.d, k = static_cast<int64_t>(d.Hkv) * d.d;
  const Span read[] = {{"dQr", dQr, t, q, q}, {"dKr", dKr, t, k, k}, {"Q", Q, t, d.qs, q}, {"K", K, t, d.ks, k},
                       flat("inv_freq", inv_freq, d.rot / 2, 4), flat("q_weight", q_weight, d.d, 4),
                       flat("k_weight", k_weight, d.d, 4), flat("pos", pos, t, 4)};
  const Span out[] = {{"dQ", dQ, t, q, q}, {"dK", dK, t, k, k}, flat("dq_weight", dq_weight, d.d, 4),
                      flat("dk_weight", dk_weight, d.d, 4), flat("workspace", ws, static_cast<int64_t>(pisa::rope_bwd_ws(d)), 1)};
  PISA_CHECK(check_apart(read, out, 2));
  return cuda_rc(pisa::launch_rope_bwd(d, Q, K, dQr, dKr, inv_freq, q_weight, k_weight, pos, dQ, dK, dq_weight,
                                       dk_weight, static_cast<char*>(ws), stream),
                 "pisa_qk_norm_rope_bwd");
}

}  // extern "C"
