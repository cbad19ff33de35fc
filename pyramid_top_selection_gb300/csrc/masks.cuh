// What the rows of the tensor-core attention see, and what becomes of their scores: a window with sinks, or the document
// that a row belongs to, with scores as they are or capped and biased by distance. The forward and backward kernels
// (window_fwd.cuh, window_bwd.cuh) take one of these as a template argument.
#pragma once

#include "scores.cuh"
#include "window_tc.cuh"

namespace pisa {
namespace win {

// (flags: kDocs, with capped scores, with scores that lose a slope times the distance)
constexpr int kWindow = 0, kDocs = 1, kCap = 2, kBias = 4;
// (and kSearch: documents looked up among the starts, not in a table. A flag, for the search in line cost the capped forward of
// long documents 7 % of its time, whether it was run or not.)
constexpr int kSearch = 8;

// Documents on the device. Where there are many tokens, a kernel laid their rows out before (doc_rows.cuh).
struct DocRows {
  const int4* bounds;      // [T + 1], of() of every token; not with kSearch
  const int32_t* order;    // token tiles, those with the most keys first; not with kSearch
  const int32_t* key_order;   // tiles of 128 keys, those with the most tokens first; for the backward
  const float* slopes;     // per query head, or NULL
  float cap;               // 0: none
  int32_t T, n_docs;
  const int32_t *starts, *prefix;

  // What is known of token t: its document's tokens [x, y), one past its prefix z (x = y = z, at the first document's
  // first token or one past the last one's: none). Of t = T: x the first document's first token, y one past the last one's.
  template <int MASK>
  __device__ __forceinline__ int4 of(int t) const {
    if constexpr (MASK & kSearch) {
      if (t == T) return make_int4(clamped(starts[0]), clamped(starts[n_docs]), 0, 0);
      return search(t, [&](int m) { return __ldg(starts + m); });
    } else {
      return bounds[t];
    }
  }
  __device__ __forceinline__ int clamped(int v) const { return max(0, min(v, T)); }
  template <class S>
  __device__ __forceinline__ int4 search(int t, S start_of) const {
    int lo = 0, hi = n_docs + 1;                       // starts below lo are <= t, those from hi on are > t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (start_of(mid) <= t) lo = mid + 1; else hi = mid;
    }
    int4 b;
    if (lo == 0 || lo > n_docs) {
      b.x = b.y = b.z = clamped(start_of(lo == 0 ? 0 : n_docs));
    } else {
      b.x = clamped(start_of(lo - 1));
      b.y = clamped(start_of(lo));
      b.z = prefix ? b.x + max(0, min(__ldg(prefix + lo - 1), b.y - b.x)) : b.x;
    }
    b.w = 0;
    return b;
  }
};

// The keys [lo, hi] that token t sees (hi < lo: none).
template <int MASK>
struct DocSpan {
  int lo, hi;
  __device__ __forceinline__ DocSpan() : lo(0), hi(-1) {}
  __device__ __forceinline__ DocSpan(const DocRows& d, int t) {
    const int4 b = d.of<MASK>(t);
    lo = b.x;
    hi = t < b.y ? max(t, b.z - 1) : -1;
  }
};

// The keys [lo, hi] that some token of [t0, t1) sees: spans neither begin nor end before an earlier token's.
template <int MASK>
struct DocRange {
  int lo, hi;
  __device__ __forceinline__ DocRange(const DocRows& d, int t0, int t1) : lo(0), hi(-1) {
    if (t0 >= t1) return;
    const int4 a = d.of<MASK>(t0), z = d.of<MASK>(t1 - 1);
    lo = a.x;
    hi = t1 - 1 < z.y ? max(t1 - 1, z.z - 1) : z.y - 1;
  }
};

// The tokens [first, end) that see key j.
struct DocSeen {
  int first, end;
  __device__ __forceinline__ DocSeen(const DocRows& d, int j, int T) : first(0), end(0) {
    if (j >= T) return;
    const int4 b = d.bounds[j];
    if (j >= b.y || j < b.x) return;
    first = j < b.z ? b.x : j;
    end = b.y;
  }
};

// Scores in powers of two from a thread's products x, before the distance's share:
//   y = scale log2 e x, or (CAP) cap log2 e tanh(k x), k = scale / cap. Where a warp has no product beyond |k x| = 3/4, tanh
//   is a polynomial of (k x)^2 on the FMA units (minimax, within 2.7e-7 in fp32), its coefficients taken times k^2i and
//   scale log2 e: 6 operations; else 1 - 2 / (1 + e^(2 k x)) (within 2.5e-7): 3 of the FMA units and two special
//   functions, of which the reciprocal alone takes as long as the 6 (16 a cycle and SM).
// Not hidden by the products, though no unit is full (in the capped forward FMA 21-23 %, ALU 20 %, special functions 21 %, issue slots 40-43
// %): they lengthen a tile's chain from tensor memory over the cap, the maximum and the exponentials to P, and two softmax warps a
// scheduler do not hide it.
template <bool CAP>
struct Scores {
  float k, cap2, back2;    // scale / cap, cap log2 e, -1 / (cap log2 e)^2
  uint64_t p[CAP ? 5 : 1]; // coefficients in pairs (p[0] alone: scale log2 e)
  __device__ __forceinline__ Scores(float scale, float cap) : k(0.f), cap2(0.f), back2(0.f) {
    const float c1 = scale * kScoreLog2e;
    p[0] = tc::pack2(c1, c1);
    if (CAP) {
      k = scale / cap;
      cap2 = cap * kScoreLog2e;
      back2 = -1.f / (cap2 * cap2);
      const float k2 = k * k, c[5] = {0.999997199f, -0.333230764f, 0.132260919f, -0.0492804497f, 0.0123188347f};
      float f = c1;
#pragma unroll
      for (int i = 0; i < 5; ++i, f *= k2) p[CAP ? i : 0] = tc::pack2(c[i] * f, c[i] * f);
    }
  }
  // N products to y, in place; the chains of four pairs side by side.
  template <int N>
  __device__ __forceinline__ void apply(float (&x)[N]) const { apply_with<false>(x, [](int) { return 0.f; }); }
  // The same plus add(q) for the q-th 16 of them.
  template <int N, class A>
  __device__ __forceinline__ void apply(float (&x)[N], A add) const { apply_with<true>(x, add); }

 private:
  template <bool ADD, int N, class A>
  __device__ __forceinline__ void apply_with(float (&x)[N], A add) const {
    auto plus = [&](uint64_t a, uint64_t b, int c) {           // a b, plus what is added at column c
      if constexpr (!ADD) return mul2(a, b);
      const float s = add(c >> 4);
      return tc::fma2(a, b, tc::pack2(s, s));
    };
    if constexpr (!CAP) {
#pragma unroll
      for (int c = 0; c < N; c += 2) tc::unpack2(plus(tc::pack2(x[c], x[c + 1]), p[0], c), x[c], x[c + 1]);
    } else {
      float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < N; c += 8)
#pragma unroll
        for (int q = 0; q < 4; ++q) asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(top[q]) : "f"(x[c + q]), "f"(x[c + 4 + q]));
      if (__all_sync(0xffffffffu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * k <= 0.75f)) {
#pragma unroll
        for (int c0 = 0; c0 < N; c0 += 8) {
          uint64_t v[4], r[4], y[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            v[c] = tc::pack2(x[c0 + 2 * c], x[c0 + 2 * c + 1]);
            y[c] = mul2(v[c], v[c]);
            r[c] = p[4];
          }
#pragma unroll
          for (int i = 3; i >= 0; --i)
#pragma unroll
            for (int c = 0; c < 4; ++c) r[c] = tc::fma2(r[c], y[c], p[i]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::unpack2(plus(v[c], r[c], c0 + 2 * c), x[c0 + 2 * c], x[c0 + 2 * c + 1]);
        }
      } else {
        const float e2 = 2.f * kScoreLog2e * k;
        const uint64_t ee = tc::pack2(e2, e2), one = tc::pack2(1.f, 1.f), m2 = tc::pack2(-2.f * cap2, -2.f * cap2);
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          float a, b;
          tc::unpack2(mul2(tc::pack2(x[c], x[c + 1]), ee), a, b);
          tc::unpack2(tc::add2(tc::pack2(tc::ex2(a), tc::ex2(b)), one), a, b);
          const float top = cap2 + (ADD ? add(c >> 4) : 0.f);
          tc::unpack2(tc::fma2(tc::pack2(rcp_approx(a), rcp_approx(b)), m2, tc::pack2(top, top)), x[c], x[c + 1]);
        }
      }
    }
  }

 public:
  // What a gradient takes through the cap, from capped scores: 1 - tanh^2.
  __device__ __forceinline__ uint64_t back(uint64_t y) const { return tc::fma2(mul2(y, y), tc::pack2(back2, back2), tc::pack2(1.f, 1.f)); }
};

// 128 consecutive fp32 columns of this thread's TMEM lane, in one load.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
  uint32_t r[128];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,"
      "%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
      "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,"
      "%88,%89,%90,%91,%92,%93,%94,%95,%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]), "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int k = 0; k < 128; ++k) v[k] = __uint_as_float(r[k]);
}

// The distance's share of a row's scores against columns 0 .. N - 1 of a tile, powers of two: -slope |d0 - c|, d0 the row's
// position less the first column's key. Where a row sees no later key, -slope (d0 - c): linear in c, as a term of
// each 16 columns, which costs nothing where it goes into another sum, and one of 16 that do not change.
struct Distance {
  float slope;
  uint64_t part[8];        // slope c, c = 0 .. 15, in pairs
  bool ahead;              // some row of the warp sees later keys
  __device__ __forceinline__ void set(float slope_, bool sees_later) {
    slope = slope_;
    ahead = __any_sync(0xffffffffu, sees_later);
#pragma unroll
    for (int c = 0; c < 8; ++c) part[c] = tc::pack2(slope * (2 * c), slope * (2 * c + 1));
  }
  __device__ __forceinline__ float base(float d0, int c16) const { return -slope * (d0 - static_cast<float>(c16)); }
};

}  // namespace win
}  // namespace pisa
