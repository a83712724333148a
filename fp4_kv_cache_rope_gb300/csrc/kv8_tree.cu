// Attention of drafted tokens: what the cached rows gave a query is joined with the
// drafted rows on its path to the root, which are no rows of the cache.
//
//   o = (sum_parts 2^(m_p - m) o_p + sum_path 2^(x_a - m) v_a) / (... the sums alike)
//
// A drafted tree's path is a handful of rows, so they are taken one by one: eight lanes
// a row, fp32 throughout.  The cached rows' part, which is where the bytes are, comes
// from the kernels that attend over the cache.
//
// Latency bounds it: lengths, the walk to the root, the parts, then a path row after
// another.  Trees of 60 tokens of 16 sequences, 32 heads, D 128 (up to 30,720 query
// rows): 24 us on cold caches, of 137 us for the call.  The work grows with the paths'
// rows in all, so chains, which kv8_attn takes too once they are in the cache, pay for their
// squares: 256 tokens of the 16 sequences take 1424 us where none follows another takes 425
// us and a random tree (paths up to 21) 476 us.
#include "kv8_tree.cuh"
#include "kv8_scores.cuh"

namespace csa2 {
namespace {

struct JoinParams {
  Kv8Attn a;
  Kv8Scores sc;
  Kv8Left left;
  Kv8Rows k, v;            // the drafted rows [B, T, kv_heads, D]
};

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kPreRows = 256;              // query rows of a CTA of the many-row kernel

// Eight lanes' share of a 16-bit row: chunks lane and lane + 8 of eight channels (D
// 64: one).
template <int D>
struct Share {
  static constexpr int kCh = D / 8;
  float v[kCh];
  __device__ __forceinline__ void take(const uint4 (&raw)[D / 64], int type) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (type == CSA2_BF16) {
          bf16x2_to_f32(w[i], v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          v[8 * c + 2 * i] = f.x;
          v[8 * c + 2 * i + 1] = f.y;
        }
      }
    }
  }
  __device__ __forceinline__ void load(const Kv8Rows& r, int64_t at, int l8) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(r.data) + 2 * at) + l8;
    uint4 raw[D / 64];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) raw[c] = p[8 * c];
    take(raw, r.type);
  }
  __device__ __forceinline__ void load(const float* row, int l8) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float4*>(v + 8 * c + 4 * i) =
            *reinterpret_cast<const float4*>(row + 64 * c + 8 * l8 + 4 * i);
  }
};

template <int D>
struct Running {
  float top = -INFINITY, sum = 0.0f;
  float o[D / 8] = {};
  // (a sum of 0: nothing was seen; of NaN: the query holds one, and it stays)
  __device__ __forceinline__ void join(float m, float s, const float (&y)[D / 8]) {
    const float nt = fmaxf(top, m);
    const float f = sum == 0.0f ? 0.0f : kv8_exp2(top - nt), g = s == 0.0f ? 0.0f : kv8_exp2(m - nt);
    sum = sum * f + s * g;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i] = o[i] * f + y[i] * g;
    top = nt;
  }
};

// WIDE: a CTA's eight warps for one query row, whose parts and path their 32 groups of
// eight lanes take in turn.  Otherwise a group for a row: a token's heads lie next to
// each other, so the four groups of a warp read the same drafted rows, and nothing is
// left to put together.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kJoinThreads) kv8_tree_join_kernel(JoinParams p) {
  constexpr int kRows = WIDE ? 1 : 4 * kJoinWarps;
  __shared__ uint8_t path[kRows][CSA2_KV8_MAX_TREE];
  __shared__ float stat[2][kJoinWarps];
  __shared__ float outs[WIDE ? kJoinWarps : 1][D];
  griddep_wait();
  griddep_launch_dependents();
  const Kv8& c = p.a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l8 = lane & 7;
  const int grp = warp * 4 + (lane >> 3);
  const int64_t rows = (int64_t)c.batch * p.a.T * p.a.H;
  int64_t row = WIDE ? blockIdx.x : (int64_t)blockIdx.x * kRows + grp;   // of [B, T, H]
  bool real = row < rows;
  if (!real) row = rows - 1;
  const int hd = (int)(row % p.a.H), tok = (int)(row / p.a.H % p.a.T), b = (int)(row / p.a.H / p.a.T);
  int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
  ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
  real &= tok < ql;
  if (WIDE && !real) return;                 // (the whole CTA)
  const int n = kv8_len(c, b), h = hd / p.a.G;

  // ---- the path: itself, its parent, ..
  uint8_t* mine = path[WIDE ? 0 : grp];
  int depth = -1;
  if (real) {
    const int32_t* parent = p.sc.parent + (int64_t)b * p.a.T;
    bool bad = false;
    for (int at = tok;;) {
      ++depth;
      if (l8 == 0) mine[depth] = (uint8_t)at;
      const int up = parent[at];
      bad = up >= at;
      if (up < 0 || bad) break;
      at = up;
    }
    if (bad && l8 == 0) set_status(p.a.status, CSA2_DEV_BAD_TREE);
  }
  if (WIDE)
    __syncthreads();
  else
    __syncwarp();

  Share<D> q;
  q.load(p.a.q, b * p.a.q.sb + (int64_t)tok * p.a.q.st + (int64_t)hd * p.a.q.sh, l8);
  Running<D> all;
  const int from = WIDE ? grp : 0;
  constexpr int kStride = WIDE ? 4 * kJoinWarps : 1;

  // ---- the cached rows' parts
  int parts = 1, c0 = 0, gr = tok * p.a.G + hd % p.a.G;
  if (p.left.kind == 1) {
    // (a whole warp's work: a row of each group after another)
    const int unit = h * p.left.tiles + gr / p.left.tile_rows;
#pragma unroll 1
    for (int g = 0; g < 32; g += 8) {
      int first, last;
      kv8_sharers_by(c, lane, c.heads * p.left.tiles, p.left.ctas, __shfl_sync(0xffffffffu, b, g),
                     __shfl_sync(0xffffffffu, unit, g), first, last,
                     [&](int i) { return kv8_span<kKv8Step>(p.a, p.sc, i).steps; });
      if (WIDE || (lane & 24) == g) {
        c0 = first;
        parts = last - first + 1;
      }
      if (WIDE) break;
    }
  } else if (p.left.kind == 2) {
    parts = p.left.ctas;
  }
  if (!real) parts = 0;
  const int in = gr % max(p.left.tile_rows, 1);
#pragma unroll 2
  for (int i = from; i < parts; i += kStride) {
    const float *o, *m, *s;
    if (p.left.kind == 2) {
      const int64_t id = (((int64_t)(p.left.tiles - 1 - gr / kPreRows) * c.batch + b) * p.left.ctas + i) *
                             c.heads + h;
      const float* part = p.a.part + id * kPreRows * (D + 2);
      o = part + in * D;
      m = part + kPreRows * D + in;
      s = m + kPreRows;
    } else if (parts > 1) {
      const float* part =
          p.a.part + (2 * (int64_t)(c0 + i) + (i == 0)) * (kKv8SlotRows * (D + 2));
      o = part + in * D;
      m = part + kKv8SlotRows * D + in;
      s = m + kKv8SlotRows;
    } else {
      o = p.sc.rows_out + row * kv8_row_floats(D);
      m = o + D;
      s = m + 1;
    }
    Share<D> y;
    y.load(o, l8);
    // (the many-row kernel's weights are 2^7 times what its maximum says)
    all.join(p.left.kind == 2 ? *m - 7.0f : *m, *s, y.v);
  }

  // ---- the path's rows, the next one on its way while one is worked on
  const float slope = p.sc.slopes ? p.sc.slopes[hd] * kLog2e : 0.0f;
  const char* kp = static_cast<const char*>(p.k.data) + 2 * (b * p.k.sb + (int64_t)h * p.k.sh);
  const char* vp = static_cast<const char*>(p.v.data) + 2 * (b * p.v.sb + (int64_t)h * p.v.sh);
  constexpr int kC = D / 64;
  uint4 rk[kC], rv[kC];
  auto fetch = [&](int i) {
    const int64_t at = i <= depth ? mine[i] : 0;   // (a row that is there)
    const uint4* k = reinterpret_cast<const uint4*>(kp + 2 * at * p.k.st) + l8;
    const uint4* v = reinterpret_cast<const uint4*>(vp + 2 * at * p.v.st) + l8;
#pragma unroll
    for (int cc = 0; cc < kC; ++cc) {
      rk[cc] = k[8 * cc];
      rv[cc] = v[8 * cc];
    }
  };
  // (whole warps: the dot's shuffles)
  const int longest = __reduce_max_sync(0xffffffffu, depth);
  fetch(from);
#pragma unroll 1
  for (int i0 = 0; i0 <= longest; i0 += kStride) {
    const int i = i0 + from;
    Share<D> k, v;
    k.take(rk, p.a.q.type);
    v.take(rv, p.a.q.type);
    if (i0 + kStride <= longest) fetch(i + kStride);
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < Share<D>::kCh; ++e) dot = fmaf(q.v[e], k.v[e], dot);
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
    dot += __shfl_xor_sync(0xffffffffu, dot, 4);
    float x = dot * p.sc.factor;
    if (p.sc.cap2 > 0.0f) x = kv8_cap(x, p.sc.cap2);
    x = fmaf(-slope, (float)i, x);
    const bool ok = i <= depth && (!p.sc.window || i < p.sc.window || n + depth - i < p.sc.sink);
    if (ok && x != -INFINITY) all.join(x, 1.0f, v.v);
  }

  // ---- the groups together
  if (WIDE) {
#pragma unroll
    for (int d = 8; d < 32; d *= 2) {
      float y[D / 8];
#pragma unroll
      for (int e = 0; e < D / 8; ++e) y[e] = __shfl_xor_sync(0xffffffffu, all.o[e], d);
      const float m = __shfl_xor_sync(0xffffffffu, all.top, d);
      const float s = __shfl_xor_sync(0xffffffffu, all.sum, d);
      all.join(m, s, y);
    }
    if (lane < 8) {
#pragma unroll
      for (int cc = 0; cc < kC; ++cc)
#pragma unroll
        for (int e = 0; e < 8; ++e) outs[warp][64 * cc + 8 * l8 + e] = all.o[8 * cc + e];
      if (lane == 0) {
        stat[0][warp] = all.top;
        stat[1][warp] = all.sum;
      }
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) {
      Share<D> y;
      y.load(outs[w], l8);
      all.join(stat[0][w], stat[1][w], y.v);
    }
    real = lane < 8;
  }
  if (real) {
    const float inv = all.sum == 0.0f ? 0.0f : 1.0f / all.sum;
    uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.a.out.data)) + b * p.a.out.sb +
                    (int64_t)tok * p.a.out.st + (int64_t)hd * p.a.out.sh;
#pragma unroll
    for (int cc = 0; cc < kC; ++cc) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack16(all.o[8 * cc + 2 * e] * inv, all.o[8 * cc + 2 * e + 1] * inv, p.a.out.type);
      *reinterpret_cast<uint4*>(out + 64 * cc + 8 * l8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (p.a.lse && l8 == 0)
      p.a.lse[row] = all.sum == 0.0f ? -INFINITY : (all.top + log2f(all.sum)) * 0.6931471805599453f;
  }
}

template <int D>
cudaError_t join_as(const JoinParams& p, int num_sms, cudaStream_t s) {
  const int64_t rows = (int64_t)p.a.c.batch * p.a.T * p.a.H;
  // Few query rows: eight warps each, for the parts of a unit that many CTAs shared.  Trees
  // over 2 sequences of 8192 rows, 32 heads, D 128, the call: 8 tokens (512 rows) 27.5 us, and
  // 30.1 with a group a row; 16 tokens 44 and 37 us, 32 tokens 51 and 36 us.  (Long paths have
  // more to share: a chain of 64 tokens of 8 heads 38 and 59 us, of 128 65 and 94 us.)
  if (rows <= 4 * num_sms)
    return kv8_launch(kv8_tree_join_kernel<D, true>, dim3((unsigned)rows), kJoinThreads, 0, s, p);
  constexpr int kRows = 4 * kJoinWarps;
  return kv8_launch(kv8_tree_join_kernel<D, false>, dim3((unsigned)((rows + kRows - 1) / kRows)),
                    kJoinThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_kv8_tree_join(const Kv8Attn& a, const Kv8Scores& sc, const Kv8Left& left,
                                 const Kv8Rows& k, const Kv8Rows& v, int num_sms, cudaStream_t s) {
  const JoinParams p{a, sc, left, k, v};
  return a.D == 64 ? join_as<64>(p, num_sms, s) : join_as<128>(p, num_sms, s);
}

}  // namespace csa2
