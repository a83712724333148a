// The position rotation of query and key rows, the 8-bit cache's append with it,
// and the append of chosen rows.
//
//   (x0, x1) -> (x0 c - x1 s, x0 s + x1 c),   (c, s) = table[position][pair]
//
// with each product and sum rounded once in fp32, so that the bytes do not depend
// on how the work was shared out.  A thread takes two 16-byte chunks of eight
// channels that rotate against each other (CSA2_ROPE_HALVES) or each within itself
// (CSA2_ROPE_PAIRS); either way it needs the eight (c, s) from pair 8 u on.  The
// chunks that are not rotated go two to a thread as well.
//
// All of it moves bytes: the rows once in, once out.
#include "kv8_append.cuh"
#include "kv8_tree.cuh"

namespace csa2 {
namespace {

struct RopeTable {
  const float *cos, *sin;
  int32_t positions, dim, first, style;
};

// The two chunks of thread u of a row's D / 16, and whether they are rotated.
struct Chunks {
  int a, b;
  bool on;
};
template <int D>
__device__ __forceinline__ Chunks chunks_of(const RopeTable& r, int u) {
  const int n = r.dim >> 4, f = r.first >> 3;       // rotated threads, first rotated chunk
  Chunks c;
  c.on = u < n;
  if (c.on) {
    c.a = r.style == CSA2_ROPE_HALVES ? f + u : f + 2 * u;
    c.b = r.style == CSA2_ROPE_HALVES ? c.a + n : c.a + 1;
  } else {
    const int e = 2 * (u - n);                      // of the others in order
    c.a = e < f ? e : e + 2 * n;
    c.b = e + 1 < f ? e + 1 : e + 1 + 2 * n;
  }
  return c;
}

// Eight channels: 16 bytes, or 32 of fp32.
template <int TYPE>
struct Eight {
  uint4 w[TYPE == CSA2_F32 ? 2 : 1];
  __device__ __forceinline__ void zero() {
    w[0] = make_uint4(0, 0, 0, 0);
    if (TYPE == CSA2_F32) w[TYPE == CSA2_F32] = w[0];
  }
  __device__ __forceinline__ void load(const char* row, int chunk) {
    const uint4* p = reinterpret_cast<const uint4*>(row + chunk * (TYPE == CSA2_F32 ? 32 : 16));
    w[0] = p[0];
    if (TYPE == CSA2_F32) w[TYPE == CSA2_F32] = p[1];
  }
  __device__ __forceinline__ void store(char* row, int chunk) const {
    uint4* p = reinterpret_cast<uint4*>(row + chunk * (TYPE == CSA2_F32 ? 32 : 16));
    p[0] = w[0];
    if (TYPE == CSA2_F32) p[1] = w[TYPE == CSA2_F32];
  }
  __device__ __forceinline__ void to(float (&v)[8]) const {
    const uint32_t* x = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == CSA2_F32) {
        v[2 * i] = __uint_as_float(x[2 * i]);
        v[2 * i + 1] = __uint_as_float(x[2 * i + 1]);
      } else if (TYPE == CSA2_BF16) {
        bf16x2_to_f32(x[i], v[2 * i], v[2 * i + 1]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void from(const float (&v)[8]) {
    uint32_t* x = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == CSA2_F32) {
        x[2 * i] = __float_as_uint(v[2 * i]);
        x[2 * i + 1] = __float_as_uint(v[2 * i + 1]);
      } else {
        x[i] = pack16(v[2 * i], v[2 * i + 1], TYPE);
      }
    }
  }
};

struct Turn {            // the cosines and sines of a thread's pairs
  float c[8], s[8];
};
__device__ __forceinline__ Turn turn_at(const RopeTable& r, const Chunks& k, int u, int pos) {
  Turn t;
  if (k.on && pos >= 0 && pos < r.positions) {
    const int64_t at = (int64_t)pos * (r.dim >> 1) + 8 * u;
    const float4* c = reinterpret_cast<const float4*>(r.cos + at);
    const float4* s = reinterpret_cast<const float4*>(r.sin + at);
    *reinterpret_cast<float4*>(t.c) = c[0];
    *reinterpret_cast<float4*>(t.c + 4) = c[1];
    *reinterpret_cast<float4*>(t.s) = s[0];
    *reinterpret_cast<float4*>(t.s + 4) = s[1];
  }
  return t;
}
// (Single operations: the packed product and sum are contracted into one that rounds once.)
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(x, s), __fmul_rn(y, c));
  x = a;
}
__device__ __forceinline__ void turn_rows(float (&a)[8], float (&b)[8], const Turn& t, int style) {
  if (style == CSA2_ROPE_HALVES) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], t.c[i], t.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn_pair(a[2 * i], a[2 * i + 1], t.c[i], t.s[i]);
      turn_pair(b[2 * i], b[2 * i + 1], t.c[4 + i], t.s[4 + i]);
    }
  }
}

// ------------------------------------------------------- rows outside the cache
struct RopeParams {
  Kv8 c;
  RopeTable r;
  Kv8Rows in[2], out[2];   // queries, keys
  int32_t heads[2];
  int32_t T;
  const int32_t* len;      // [B] or null (= T)
  const int32_t* start;    // [B] or null (= seq_len)
  const int32_t* pos;      // [B, T] or null
  const int32_t* parent;   // [B, T] or null
  uint32_t* status;
};

__device__ __forceinline__ char* row_at(const Kv8Rows& r, int es, int b, int tok, int h) {
  return static_cast<char*>(const_cast<void*>(r.data)) + (b * r.sb + (int64_t)tok * r.st + h * r.sh) * es;
}

// One CTA per token, D / 16 threads a row.  A thread's cosines and sines serve all
// heads of the token; its first row is on its way while the position is looked up.
// Bound by HBM: 16,384 tokens of 64 query and 8 key heads, D 128, bf16: 612 MB in 95 us,
// 6.4 TB/s.  What counts is how many CTAs wait for memory at once: six an SM with one
// row a thread in flight, where three with three rows took 104 us and four 99 us.
constexpr int kRopeThreads = 256;
template <int D, int TYPE>
__global__ void __launch_bounds__(kRopeThreads, TYPE == CSA2_F32 ? 4 : 6) kv8_rope_kernel(RopeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kLanes = D / 16, kSize = TYPE == CSA2_F32 ? 4 : 2;
  const int b = blockIdx.y, tok = blockIdx.x;
  int t = p.len ? p.len[b] : p.T;
  t = t < 0 ? 0 : (t > p.T ? p.T : t);
  if (tok >= t) return;
  const int u = threadIdx.x % kLanes, sub = threadIdx.x / kLanes, rows = blockDim.x / kLanes;
  const int all = p.heads[0] + p.heads[1];
  Chunks k = chunks_of<D>(p.r, u);
  Eight<TYPE> x, y;
  auto load = [&](int h) {
    const int set = h >= p.heads[0];
    const char* from = row_at(p.in[set], kSize, b, tok, set ? h - p.heads[0] : h);
    x.load(from, k.a);
    y.load(from, k.b);
  };
  if (sub < all) load(sub);
  int at;
  if (p.pos) {
    at = p.pos[(int64_t)b * p.T + tok];
  } else {
    at = p.start ? min(p.start[b], 1 << 30) : kv8_len(p.c, b);
    if (p.parent) {
      bool bad = false;
      at += kv8_depth(p.parent + (int64_t)b * p.T, tok, bad);
      if (bad && threadIdx.x == 0) set_status(p.status, CSA2_DEV_BAD_TREE);
    } else {
      at += tok;
    }
  }
  const bool inside = at >= 0 && at < p.r.positions;
  if (!inside && threadIdx.x == 0) set_status(p.status, CSA2_DEV_BAD_INDEX);
  k.on &= inside;
  const Turn turn = turn_at(p.r, k, u, at);
  for (int h = sub; h < all; h += rows) {
    if (h > sub) load(h);
    if (k.on) {
      float v[8], w[8];
      x.to(v);
      y.to(w);
      turn_rows(v, w, turn, p.r.style);
      x.from(v);
      y.from(w);
    }
    const int set = h >= p.heads[0];
    char* to = row_at(p.out[set], kSize, b, tok, set ? h - p.heads[0] : h);
    x.store(to, k.a);
    y.store(to, k.b);
  }
}

template <int D>
cudaError_t rope_of(const RopeParams& p, cudaStream_t s) {
  // as few threads as need no more passes
  const int items = (p.heads[0] + p.heads[1]) * (D / 16);
  const int passes = (items + kRopeThreads - 1) / kRopeThreads;
  const int threads = ((items + passes - 1) / passes + 31) / 32 * 32;
  const dim3 grid(p.T, p.c.batch);
  const int type = p.in[0].type;
  auto kern = type == CSA2_F32    ? kv8_rope_kernel<D, CSA2_F32>
              : type == CSA2_BF16 ? kv8_rope_kernel<D, CSA2_BF16>
                                  : kv8_rope_kernel<D, CSA2_F16>;
  return kv8_launch(kern, grid, threads, 0, s, p);
}

// ------------------------------------------------------------ rows into the cache
struct AppendRopeParams {
  AppendParams a;          // K and V
  RopeTable r;
  const int32_t* pos;      // [B, T] or null
  Kv8Rows q, q_out;
  int32_t q_heads;
};

__device__ __forceinline__ int rope_position(const AppendRopeParams& p, const Span& sp, int b, int i) {
  return p.pos ? p.pos[(int64_t)b * p.a.T + i] : sp.first + i;
}

// The new K rows of one block and head, rotated and held in fp32 between the
// block's maximum and their codes, by NT threads.
template <int D, int TYPE, int NT, int PASSES>
struct TurnedRows {
  static constexpr int kLanes = D / 16;
  static constexpr int kRows = NT / kLanes;
  float v[PASSES][2][8];
  float s0;

  __device__ __forceinline__ void read(const AppendRopeParams& p, const Span& sp, int b, int h, int lo,
                                       int hi, bool had, const float* scale, int tid, Chunks& k) {
    const int u = tid % kLanes, sub = tid / kLanes;
    k = chunks_of<D>(p.r, u);
    s0 = had ? *scale : 0.0f;
    // Everything is asked for before anything is used, up to two rows' tables at a time.
    constexpr int kAhead = PASSES < 2 ? PASSES : 2;
    Eight<TYPE> x[PASSES], y[PASSES];
    Turn turn[kAhead];
    bool on[kAhead];
    auto look_up = [&](int i) {
      const int at = lo + i * kRows + sub;
      on[i % kAhead] = false;
      if (i >= PASSES || at >= hi) return;
      const int pos = rope_position(p, sp, b, at - sp.start);
      if (pos < 0 || pos >= p.r.positions) {
        if (u == 0) set_status(p.a.status, CSA2_DEV_BAD_INDEX);
        return;
      }
      on[i % kAhead] = k.on;
      turn[i % kAhead] = turn_at(p.r, k, u, pos);
    };
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int at = lo + i * kRows + sub;
      x[i].zero();
      y[i].zero();
      if (at < hi) {
        const char* from = row_at(p.a.in[0], TYPE == CSA2_F32 ? 4 : 2, b, at - sp.start, h);
        x[i].load(from, k.a);
        y[i].load(from, k.b);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) look_up(i);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      x[i].to(v[i][0]);
      y[i].to(v[i][1]);
      if (on[i % kAhead]) turn_rows(v[i][0], v[i][1], turn[i % kAhead], p.r.style);
      if (i + kAhead < PASSES) look_up(i + kAhead);
    }
  }

  template <int FMT>
  __device__ __forceinline__ void write(const AppendRopeParams& p, uint8_t* codes, float* scale,
                                        int64_t row0, int b0, int lo, int hi, uint32_t* red, int tid,
                                        const Chunks& k) {
    const int sub = tid / kLanes;
    constexpr uint32_t kInf = 0x7F800000u;
    float top = 0.0f;                      // a NaN stays one
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 2) top = max3_abs_nan(top, v[i][e >> 3][e & 7], v[i][e >> 3][(e & 7) + 1]);
    uint32_t bits = group_max<NT>(__float_as_uint(top), red, tid);
    const bool odd = bits >= kInf;         // uniform over the group
    if (odd) {                             // the maximum of the finite values then
      if (tid == 0) set_status(p.a.status, CSA2_DEV_NONFINITE);
      bits = 0;
#pragma unroll
      for (int i = 0; i < PASSES; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t m = __float_as_uint(v[i][e >> 3][e & 7]) & 0x7FFFFFFFu;
          if (m < kInf) bits = max(bits, m);
        }
      bits = group_max<NT>(bits, red, tid);
    }
    __syncwarp();                          // every thread of the group has read s0
    const float s1 = fmaxf(s0, kv8_scale_of<FMT>(__uint_as_float(bits)));
    const float inv = kv8_inverse(s1);
    uint8_t* dst = codes + (row0 + (lo - b0) + sub) * D;
    const uint64_t by = kv8_pair(inv, inv);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      if (lo + i * kRows + sub >= hi) continue;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) kv8_split(kv8_mul2(kv8_pair(v[i][c][e], v[i][c][e + 1]), by), x[e], x[e + 1]);
        if (odd) {                         // infinities to the largest code, NaN to 0
          constexpr float kBig = FMT == CSA2_KV8_E4M3 ? 448.0f : 127.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] != x[e] ? 0.0f : fminf(fmaxf(x[e], -kBig), kBig);
        }
        *reinterpret_cast<uint2*>(dst + (int64_t)i * kRows * D + 8 * (c ? k.b : k.a)) =
            make_uint2(kv8_encode4<FMT>(x[0], x[1], x[2], x[3]), kv8_encode4<FMT>(x[4], x[5], x[6], x[7]));
      }
    }
    block_rescale<D, FMT, NT>(codes, scale, s0, s1, inv, row0, lo - b0, tid);
  }
};

// The part of append_block for rotated K.
template <int D, int TYPE, int FMT, int NT, int PASSES>
__device__ __forceinline__ void append_turned(const AppendRopeParams& p, const Span& sp, int b, int h,
                                              int blk, uint32_t* red, int tid) {
  const Kv8& c = p.a.c;
  const int b0 = blk << c.block_shift;
  const int lo = max(sp.start, b0), hi = min(sp.start + sp.t, b0 + (1 << c.block_shift));
  if (lo >= hi) return;                    // uniform over the group
  int in_page;
  const int page = kv8_page(c, b, b0, in_page);
  if (page < 0) {
    if (tid == 0) set_status(p.a.status, CSA2_DEV_BAD_PAGE);
    return;
  }
  const int64_t row0 = kv8_row(c, page, h, in_page), at = kv8_block(c, page, h, in_page);
  TurnedRows<D, TYPE, NT, PASSES> x;
  Chunks k;
  x.read(p, sp, b, h, lo, hi, sp.start > b0, c.scales[0] + at, tid, k);
  x.template write<FMT>(p, c.codes[0], c.scales[0] + at, row0, b0, lo, hi, red, tid, k);
  if (c.mass)
    for (int r = tid; r < hi - lo; r += NT) c.mass[row0 + (lo - b0) + r] = 0.0f;
}

// 32 / (D / 16) query rows from row `at` of a sequence's t * heads on (a warp).
template <int D, int TYPE>
__device__ __forceinline__ void turn_queries(const AppendRopeParams& p, const Span& sp, int b, int at,
                                             int rows, int lane) {
  constexpr int kLanes = D / 16;
  const int row = at + lane / kLanes, u = lane % kLanes;
  if (row >= rows) return;
  const int tok = row / p.q_heads, h = row % p.q_heads;
  const int pos = rope_position(p, sp, b, tok);
  Chunks k = chunks_of<D>(p.r, u);
  if (pos < 0 || pos >= p.r.positions) {
    k.on = false;
    if (u == 0) set_status(p.a.status, CSA2_DEV_BAD_INDEX);
  }
  constexpr int kSize = TYPE == CSA2_F32 ? 4 : 2;
  const char* from = row_at(p.q, kSize, b, tok, h);
  Eight<TYPE> x, y;
  x.load(from, k.a);
  y.load(from, k.b);
  if (k.on) {
    const Turn t = turn_at(p.r, k, u, pos);
    float v[8], w[8];
    x.to(v);
    y.to(w);
    turn_rows(v, w, t, p.r.style);
    x.from(v);
    y.from(w);
  }
  char* to = row_at(p.q_out, kSize, b, tok, h);
  x.store(to, k.a);
  y.store(to, k.b);
}

// A few rows: one CTA per sequence for its keys, values and queries, a warp per
// (head, side) or four (D 64: eight) query rows, so that one launch also advances
// seq_len.  Latency: a token of 32 sequences, 64 query and 8 key heads, takes 4.4 us, and
// 1.3 MB moves.  (At D 128 its 128 registers spill 112 bytes, 248 for fp32 rows.)
template <int D, int TYPE, int FMT>
__global__ void __launch_bounds__(512) kv8_append_rope_few_kernel(AppendRopeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const Span sp = append_span(p.a, b);
  __syncthreads();
  if (threadIdx.x == 0) {
    if (sp.over) set_status(p.a.status, CSA2_DEV_OVERFLOW);
    p.a.c.seq_len[b] = sp.start + sp.t;
  }
  // (queries of rows that found no place are rotated too)
  const int turned = sp.given * p.q_heads, per = 32 / (D / 16);
  const int sides = sp.t ? 2 * p.a.c.heads : 0;
  const int first = sp.start >> p.a.c.block_shift, last = (sp.start + sp.t - 1) >> p.a.c.block_shift;
  for (int i = threadIdx.x >> 5; i < sides + (turned + per - 1) / per; i += warps) {
    if (i >= sides) {
      const int at = (i - sides) * per;
      if (p.q.type == CSA2_BF16) turn_queries<D, CSA2_BF16>(p, sp, b, at, turned, lane);
      else if (p.q.type == CSA2_F16) turn_queries<D, CSA2_F16>(p, sp, b, at, turned, lane);
      else turn_queries<D, CSA2_F32>(p, sp, b, at, turned, lane);
      continue;
    }
    for (int blk = first; blk <= last; ++blk) {
      if (i & 1)
        append_block<D, TYPE, FMT, 32, kFewRows * D / NewRows<D, TYPE, 32, 1>::EL / 32, 1, false>(
            p.a, sp, b, i >> 1, 1, blk, nullptr, lane);
      else
        append_turned<D, TYPE, FMT, 32, kFewRows * (D / 16) / 32>(p, sp, b, i >> 1, blk, nullptr, lane);
    }
  }
}

// Longer ones: one CTA per (block, head, side, sequence).  ROWS: of a block.  Four
// prompts of up to 8,192 rows, 8 heads, D 128, blocks of 64: 41 us for 145 MB and, from L2,
// 512 bytes of tables for each row and head; the instructions of the rotation (half of
// the issue slots) and the loads that wait for the lengths bound it.  Their queries (64
// heads) follow in a launch of the kernel above: 160 us in all for 921 MB, 5.8 TB/s.
template <int D, int TYPE, int FMT, int ROWS>
__global__ void __launch_bounds__(kAppendThreads, ROWS <= 64 ? 4 : 2)
    kv8_append_rope_kernel(AppendRopeParams p) {
  __shared__ uint32_t red[kAppendThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z;
  const Span sp = append_span(p.a, b);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (sp.over) set_status(p.a.status, CSA2_DEV_OVERFLOW);
    if (p.a.own_len) p.a.c.seq_len[b] = sp.start + sp.t;
  }
  if (sp.t == 0) return;
  const int blk = (sp.start >> p.a.c.block_shift) + blockIdx.x, h = blockIdx.y >> 1;
  constexpr int kPlain = ROWS * D / (TYPE == CSA2_F32 ? 4 : 8) / kAppendThreads;
  constexpr int kTurned = ROWS * (D / 16) / kAppendThreads;
  if (blockIdx.y & 1)
    append_block<D, TYPE, FMT, kAppendThreads, kPlain < 1 ? 1 : kPlain, 1, false>(p.a, sp, b, h, 1, blk,
                                                                                 red, threadIdx.x);
  else
    append_turned<D, TYPE, FMT, kAppendThreads, kTurned < 1 ? 1 : kTurned>(p, sp, b, h, blk, red,
                                                                           threadIdx.x);
}

template <int D, int TYPE, int FMT>
cudaError_t append_rope_as(AppendRopeParams p, cudaStream_t s) {
  if (p.a.T <= kFewRows)
    return kv8_launch(kv8_append_rope_few_kernel<D, TYPE, FMT>, dim3(p.a.c.batch), 512, 0, s, p);
  const int block = 1 << p.a.c.block_shift;
  p.a.own_len = p.a.start != nullptr && p.a.start != p.a.c.seq_len;
  const dim3 grid((p.a.T + block - 2) / block + 1, 2 * p.a.c.heads, p.a.c.batch);
  auto kern = block == 128  ? kv8_append_rope_kernel<D, TYPE, FMT, 128>
              : block == 64 ? kv8_append_rope_kernel<D, TYPE, FMT, 64>
                            : kv8_append_rope_kernel<D, TYPE, FMT, 32>;
  cudaError_t e = kv8_launch(kern, grid, kAppendThreads, 0, s, p);
  if (e == cudaSuccess && p.q_heads) {
    // with a start of its own it does not read the seq_len that the kernel above writes
    RopeParams r{};
    r.c = p.a.c;
    r.r = p.r;
    r.in[0] = p.q;
    r.out[0] = p.q_out;
    r.heads[0] = p.q_heads;
    r.T = p.a.T;
    r.len = p.a.new_len;
    r.start = p.a.start;
    r.pos = p.pos;
    r.status = p.a.status;
    e = rope_of<D>(r, s);
  }
  if (e != cudaSuccess || p.a.own_len) return e;
  return kv8_launch(kv8_advance_kernel, dim3((p.a.c.batch + 127) / 128), 128, 0, s, p.a);
}
template <int D, int FMT>
cudaError_t append_rope_of(const AppendRopeParams& p, cudaStream_t s) {
  return p.a.in[0].type == CSA2_F32    ? append_rope_as<D, CSA2_F32, FMT>(p, s)
         : p.a.in[0].type == CSA2_BF16 ? append_rope_as<D, CSA2_BF16, FMT>(p, s)
                                       : append_rope_as<D, CSA2_F16, FMT>(p, s);
}

RopeTable table_of(const csa2_rope& r) {
  return RopeTable{r.cos, r.sin, r.positions, r.dim, r.first, r.style};
}

}  // namespace

cudaError_t launch_kv8_rope(const Kv8& c, int D, const csa2_rope& rope, const Kv8Rows& q, int H,
                            const Kv8Rows& q_out, const Kv8Rows& k, const Kv8Rows& k_out, int T,
                            const int32_t* q_len, const int32_t* pos, const int32_t* parent,
                            uint32_t* status, cudaStream_t s) {
  const RopeParams p{c,     table_of(rope), {q, k}, {q_out, k_out}, {H, k.data ? c.heads : 0},
                     T,     q_len,          nullptr, pos,           parent,
                     status};
  return D == 64 ? rope_of<64>(p, s) : rope_of<128>(p, s);
}

cudaError_t launch_kv8_append_rope(const Kv8& c, int D, const csa2_rope& rope, const Kv8Rows& k,
                                   const Kv8Rows& v, int T, const Kv8Rows& q, int H,
                                   const Kv8Rows& q_out, const int32_t* new_len,
                                   const int32_t* start, const int32_t* pos, uint32_t* status,
                                   cudaStream_t s) {
  const AppendRopeParams p{{c, {k, v}, T, new_len, start, status, 0, nullptr, 0},
                           table_of(rope), pos, q, q_out, H};
  if (c.format == CSA2_KV8_E4M3)
    return D == 64 ? append_rope_of<64, CSA2_KV8_E4M3>(p, s) : append_rope_of<128, CSA2_KV8_E4M3>(p, s);
  return D == 64 ? append_rope_of<64, CSA2_KV8_INT8>(p, s) : append_rope_of<128, CSA2_KV8_INT8>(p, s);
}

cudaError_t launch_kv8_append_path(const Kv8& c, int D, const Kv8Rows& k, const Kv8Rows& v, int T,
                                   const int32_t* path, int M, const int32_t* new_len,
                                   const int32_t* start, uint32_t* status, cudaStream_t s) {
  const AppendParams p{c, {k, v}, M, new_len, start, status, 0, path, T};
  return append_any<true>(p, D, s);
}

}  // namespace csa2
