// What changes the scores of the 8-bit cache's attention: a cap, a slope by
// distance, a window with first rows, a prefix that every query sees, and queries
// that are drafted tokens; and which of the cached rows that leaves.
//
//   x = cap tanh(c q.k / cap) - slope |p - j|
//   seen: j < n and (j <= p or j < prefix) and (no window or j > p - window or j < sink)
#pragma once

#include "kv8_tree.cuh"

namespace csa2 {

constexpr float kLog2e = 1.44269504f;
constexpr int kNoQuery = 0x40000000;      // the "position" of a row without a query
constexpr int kKv8TreeCtas = 304;         // of the many-row kernel's parts for drafted tokens
constexpr int kKv8MaxWindow = 1 << 23;    // beyond any difference of two positions

struct Kv8Scores {
  float factor;                 // of q.k: softmax scale / cap, or, without one, times log2(e)
  float cap2;                   // cap * log2(e), or 0
  int32_t window, sink;         // 0: no window (then sink is 0)
  const float* slopes;          // [H] or null
  const int32_t* prefix;        // [B] or null
  const int32_t* parent;        // [B, T]: the queries are drafted tokens; or null
  float* rows_out;              // with parent: results of whole units, kv8_row_floats each
  // For a query at position p: rows below sees() may count, those from from() on
  // and those below `sink` do.
  __device__ __forceinline__ int sees(int p, int n, int pre) const {
    return parent ? n : min(n, max(p + 1, pre));
  }
  __device__ __forceinline__ int from(int p) const { return window ? p - window + 1 : -kNoQuery; }
};
// fp32 numbers of a query row's result before the drafted rows: O, the maximum and
// the sum; rows start on 16 bytes.
__host__ __device__ constexpr int kv8_row_floats(int D) { return D + 4; }

// Position of query `tok` of a sequence's ql.  (The depth is walked where it counts.)
__device__ __forceinline__ int kv8_query_at(const Kv8Attn& a, const Kv8Scores& sc, int b, int n, int ql,
                                            int tok) {
  if (!sc.parent) return n - ql + tok;
  if (!sc.window && !sc.slopes) return n;
  bool bad = false;
  return n + kv8_depth(sc.parent + (int64_t)b * a.T, tok, bad);
}

// The steps of STEP rows of a sequence that hold the rows which any of its queries
// sees: those of the first rows, then the ones from the earliest window's on.  (At
// least one step, of which nothing may count.)
struct Kv8Span {
  int n, steps, sinks, first;
  __device__ __forceinline__ int row(int st, int step) const {
    return (st < sinks ? st : st - sinks + first) * step;
  }
};
__device__ __forceinline__ Kv8Span kv8_span_of(const Kv8Scores& sc, int p, int end, int n, int step) {
  // p: the earliest query's position; end: rows that the last one sees
  Kv8Span s;
  s.n = n;
  const int low = sc.window ? min(max(sc.from(p), 0), end) : 0;
  s.first = low / step;
  s.sinks = min((min(sc.sink, end) + step - 1) / step, s.first);
  s.steps = s.sinks + (end + step - 1) / step - s.first;
  return s;
}
template <int STEP>
__device__ __forceinline__ Kv8Span kv8_span(const Kv8Attn& a, const Kv8Scores& sc, int b) {
  const int n = kv8_len(a.c, b);
  int ql = a.q_len ? a.q_len[b] : a.T;
  ql = ql < 0 ? 0 : (ql > a.T ? a.T : ql);
  Kv8Span s = kv8_span_of(sc, sc.parent ? n : n - ql, ql ? n : 0, n, STEP);
  s.steps = max(s.steps, 1);
  return s;
}
// About the rows of the steps of a sequence, at most (host): the ends of a window and of the
// first rows add up to a step each, of which 512 rows are counted.  Only the choice of a
// kernel and of a split goes by it.
inline int64_t kv8_most_rows(const Kv8Attn& a, const Kv8Scores& sc) {
  const int64_t seen = sc.window ? (int64_t)sc.window + sc.sink + a.T + 512 : a.c.max_len;
  return seen < a.c.max_len ? seen : a.c.max_len;
}

// Splits of the cached rows for drafted tokens' queries in the many-row kernel (base
// CTAs without), into parts of 1024 rows or so at least where a sequence is full.  Their
// results are joined with the drafted rows' in any case, so the CTAs may be cut to even out
// the sequences' lengths.  kKv8TreeCtas: two a SM.  The call for 60 tokens a sequence, D 128:
// 16 ragged sequences of up to 16384 rows, 4 K/V heads of 8, 227 us (one a SM 280, three 221);
// of up to 9000 rows, 8 heads of 4, 169 us (174, 171).  Where the lengths are even one a SM
// is enough: one sequence of 65536 rows 118 us (97, 130), 16 of 9000 rows 200 us (182, 216).
inline int kv8_tree_splits(int64_t base, int64_t most_rows) {
  const int64_t most = (most_rows + 1023) / 1024, fit = kKv8TreeCtas / base;
  const int64_t n = fit < most ? fit : most;
  return n < 1 ? 1 : (int)n;
}

// Where the results of the cached rows are once the drafted ones are joined to them
// (rows_out holds those that no entry here says otherwise of).
struct Kv8Left {
  int32_t kind;                 // 0: rows_out alone; 1: shared units of the few-row kernel; 2: splits
  int32_t tiles, tile_rows;     // 1
  int32_t ctas;                 // 1: CTAs; 2: splits
};

// ------------------------------------------------------------------------ cap
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float kv8_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh(y) / y as a quotient of two polynomials in u = y^2 of degree 4, fitted to
// |y| <= 9.02 for a small relative error (4.3e-8; 3.5e-7 with fp32's roundings, 6e-8 on
// average).  Beyond, tanh is 1 in fp32.  The quotient of the odd function keeps small
// scores' relative precision, which 1 - 2 / (1 + e^2y) would not.
constexpr float kTanhEnd = 9.02f;
__device__ __forceinline__ void kv8_tanh_parts(float y, float& p, float& q) {
  const float u = y * y;
  p = fmaf(fmaf(fmaf(fmaf(1.3319012559520615e-8f, u, 2.058343670796603e-5f), u,
                     3.4940317273139954e-3f), u, 0.13379715383052826f), u, 1.0f) * y;
  q = fmaf(fmaf(fmaf(fmaf(7.761994424981822e-7f, u, 3.2830884447321296e-4f), u,
                     2.587106265127659e-2f), u, 0.46713030338287354f), u, 1.0f);
}
// A score over the cap -> cap2 tanh of it.  A NaN stays one, and an infinity is the cap.
// (A reciprocal of its own: one shared by two keys would let a hidden key's NaN, an
// infinite query times a row that is not there, spoil a visible one.)
__device__ __forceinline__ float kv8_cap(float x, float cap2) {
  float p, q;
  kv8_tanh_parts(max_nan(min_nan(x, kTanhEnd), -kTanhEnd), p, q);
  return p * (kv8_rcp(q) * cap2);
}
// Plus `add`, rounded once with the last product.
__device__ __forceinline__ float kv8_cap(float x, float cap2, float add) {
  float p, q;
  kv8_tanh_parts(max_nan(min_nan(x, kTanhEnd), -kTanhEnd), p, q);
  return fmaf(p, kv8_rcp(q) * cap2, add);
}
// The same for |score / cap| <= kTanhNear from polynomials of degree 2 (8.9e-8; 4.5e-7 with
// fp32's roundings), for logits s that `mul` takes to scores over the cap: the
// polynomials take s itself, their coefficients the factor.  Four logits of a query at a
// time, packed, two to a reciprocal: a row's logits are all finite here, or all not, and
// hidden ones are 0.  (A fit of these degrees to 2.5 has an error of 5.1e-7 before any
// rounding.  Beyond kNearMul a coefficient could be infinite; one that is lost
// to 0 belongs to a term that is, too.)
constexpr float kTanhNear = 2.0f, kNearMul = 1e6f;
struct NearCap {
  uint64_t p0, p1, p2, q1, q2, one;
  __device__ __forceinline__ NearCap(float mul, float cap2) {
    const float m2 = mul * mul, c = cap2 * mul;
    p0 = kv8_pair(c, c);
    p1 = kv8_pair(c * (m2 * 0.1096152737736702f), c * (m2 * 0.1096152737736702f));
    p2 = kv8_pair(c * (m2 * (m2 * 9.667574195191264e-4f)), c * (m2 * (m2 * 9.667574195191264e-4f)));
    q1 = kv8_pair(m2 * 0.4429476857185364f, m2 * 0.4429476857185364f);
    q2 = kv8_pair(m2 * (m2 * 1.5285835601389408e-2f), m2 * (m2 * 1.5285835601389408e-2f));
    one = kv8_pair(1.0f, 1.0f);
  }
  // a, b: two logits each -> capped, plus `add`
  __device__ __forceinline__ void operator()(uint64_t& a, uint64_t& b, uint64_t add) const {
    const uint64_t ta = kv8_mul2(a, a), tb = kv8_mul2(b, b);
    const uint64_t na = kv8_mul2(a, kv8_fma2(kv8_fma2(p2, ta, p1), ta, p0));
    const uint64_t nb = kv8_mul2(b, kv8_fma2(kv8_fma2(p2, tb, p1), tb, p0));
    const uint64_t qa = kv8_fma2(kv8_fma2(q2, ta, q1), ta, one);
    const uint64_t qb = kv8_fma2(kv8_fma2(q2, tb, q1), tb, one);
    const uint64_t q = kv8_mul2(qa, qb);
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(q));
    const uint64_t r = kv8_pair(kv8_rcp(x), kv8_rcp(y));
    a = kv8_fma2(na, kv8_mul2(qb, r), add);
    b = kv8_fma2(nb, kv8_mul2(qa, r), add);
  }
};
// ------------------------------------- split of rows over the CTAs, as kv8_share
// kv8_share and kv8_sharers_of for the steps of the spans that `span_of` gives.
struct Kv8SpanShare : Kv8Share {
  Kv8Span span;           // the first step's sequence's
};
template <class F>
__device__ __forceinline__ Kv8SpanShare kv8_share_by(const Kv8& c, int lane, int units, int max_ctas,
                                                     int cta, F span_of) {
  Kv8SpanShare r;
  int64_t total = 0;
  if (c.batch > 32) {
    int64_t all = 0;
    for (int b = lane; b < c.batch; b += 32) all += span_of(b).steps;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    total = all * units;
  }
  int64_t x = 0, before = 0, first = 0;
  for (int base = 0;; base += 32) {
    Kv8Span mine{};
    if (base + lane < c.batch) mine = span_of(base + lane);
    int incl = mine.steps;  // at most 32 * 2^14 steps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int sum = __shfl_sync(0xffffffffu, incl, 31);
    if (base == 0) {
      if (c.batch <= 32) total = (int64_t)sum * units;
      r.ctas = kv8_sharers(total, max_ctas);
      r.x = kv8_muldiv(total, cta, r.ctas);
      r.x1 = kv8_muldiv(total, cta + 1, r.ctas);
      x = r.x < total ? r.x : total - 1;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + (int64_t)incl * units > x);
    if (hit || base + 32 >= c.batch) {
      const int l = hit ? __ffs(hit) - 1 : (c.batch - 1) & 31;
      first = before + (int64_t)__shfl_sync(0xffffffffu, incl - mine.steps, l) * units;
      r.b = base + l;
      r.span.n = __shfl_sync(0xffffffffu, mine.n, l);
      r.span.steps = __shfl_sync(0xffffffffu, mine.steps, l);
      r.span.sinks = __shfl_sync(0xffffffffu, mine.sinks, l);
      r.span.first = __shfl_sync(0xffffffffu, mine.first, l);
      break;
    }
    before += (int64_t)sum * units;
  }
  r.n = r.span.n;
  r.steps = r.span.steps;
  r.unit = (int)kv8_muldiv(x - first, 1, r.steps);
  r.step = (int)(x - first - (int64_t)r.unit * r.steps);
  return r;
}
template <class F>
__device__ __forceinline__ void kv8_sharers_by(const Kv8& c, int lane, int units, int max_ctas, int b,
                                               int unit, int& c0, int& c1, F steps_of) {
  int64_t all = 0, before = 0;
  int steps = 0;
  for (int i = lane; i < c.batch; i += 32) {
    const int s = steps_of(i);
    all += s;
    if (i < b) before += s;
    if (i == b) steps = s;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
    steps += __shfl_xor_sync(0xffffffffu, steps, o);
  }
  const int64_t total = all * units, x0 = before * units + (int64_t)unit * steps;
  const int ctas = kv8_sharers(total, max_ctas);
  // CTA i has the steps from total i / ctas on: step x is that of the last i with
  // total i < (x + 1) ctas
  c0 = (int)kv8_muldiv((x0 + 1) * ctas - 1, 1, total);
  c1 = (int)kv8_muldiv((x0 + steps) * ctas - 1, 1, total);
}

}  // namespace csa2
