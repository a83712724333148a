// Attention of drafted tokens: what the cached rows gave a query is joined with the
// drafted rows on its path to the root, which are no rows of the cache.
//
//   o = (sum_parts 2^(m_p - m) o_p + sum_path 2^(x_a - m) v_a) / (... the sums alike)
//
// A path holds a handful of rows, so they are taken one by one: eight lanes a row,
// fp32 throughout.  The cached rows' part, which is where the bytes are, comes from
// the kernels that attend over the cache.
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
  __device__ __forceinline__ void load(const Kv8Rows& r, int64_t at, int l8) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(r.data) + 2 * at) + l8;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint4 w = p[8 * c];
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r.type == CSA2_BF16) {
          bf16x2_to_f32(ww[i], v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[i]));
          v[8 * c + 2 * i] = f.x;
          v[8 * c + 2 * i + 1] = f.y;
        }
      }
    }
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

// WARPS: warps of a query row.  Each group of eight lanes takes every 4 WARPS-th of
// the parts, then of the path's rows.
template <int D, int WARPS>
__global__ void __launch_bounds__(kJoinThreads) kv8_tree_join_kernel(JoinParams p) {
  constexpr int kRows = kJoinWarps / WARPS;
  __shared__ uint8_t path[kRows][CSA2_KV8_MAX_TREE];
  __shared__ float stat[2][kJoinWarps];
  __shared__ float outs[WARPS > 1 ? kJoinWarps : 1][D];
  griddep_wait();
  griddep_launch_dependents();
  const Kv8& c = p.a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l8 = lane & 7;
  const int64_t row = (int64_t)blockIdx.x * kRows + warp / WARPS;    // of [B, T, H]
  const int hd = (int)(row % p.a.H), tok = (int)(row / p.a.H % p.a.T);
  const int64_t b64 = row / p.a.H / p.a.T;
  if (b64 >= c.batch) return;                // a whole warp; WARPS > 1: the whole CTA
  const int b = (int)b64;
  int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
  ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
  if (tok >= ql) return;                     // alike
  const int n = kv8_len(c, b), h = hd / p.a.G;

  // ---- the path: itself, its parent, ..
  const int32_t* parent = p.sc.parent + (int64_t)b * p.a.T;
  uint8_t* mine = path[warp / WARPS];
  int depth = 0;
  {
    bool bad = false;
    int at = tok;
    for (;; ++depth) {
      if (lane == 0 && warp % WARPS == 0) mine[depth] = (uint8_t)at;
      const int up = parent[at];
      if (up < 0) break;
      if (up >= at) {
        bad = true;
        break;
      }
      at = up;
    }
    if (bad && lane == 0) set_status(p.a.status, CSA2_DEV_BAD_TREE);
  }
  if (WARPS > 1)
    __syncthreads();
  else
    __syncwarp();

  Share<D> q;
  q.load(p.a.q, b * p.a.q.sb + (int64_t)tok * p.a.q.st + (int64_t)hd * p.a.q.sh, l8);
  Running<D> all;
  const int grp = warp % WARPS * 4 + (lane >> 3);
  constexpr int kGroups = 4 * WARPS;

  // ---- the cached rows' parts
  int parts = 1, c0 = 0, gr = tok * p.a.G + hd % p.a.G;
  if (p.left.kind == 1) {
    int c1;
    kv8_sharers_by(c, lane, c.heads * p.left.tiles, p.left.ctas, b,
                   h * p.left.tiles + gr / p.left.tile_rows, c0, c1,
                   [&](int i) { return kv8_span<kKv8Step>(p.a, p.sc, i).steps; });
    parts = c1 - c0 + 1;
  } else if (p.left.kind == 2) {
    parts = p.left.ctas;
  }
  const int in = gr % max(p.left.tile_rows, 1);
  for (int i = grp; i < parts; i += kGroups) {
    const float *o, *m, *s;
    if (p.left.kind == 2) {
      const int64_t id =
          (((int64_t)(p.left.tiles - 1 - gr / kPreRows) * c.batch + b) * parts + i) * c.heads + h;
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

  // ---- the path's rows
  const float slope = p.sc.slopes ? p.sc.slopes[hd] * kLog2e : 0.0f;
  for (int i0 = 0; i0 <= depth; i0 += kGroups) {   // (whole warps: the dot's shuffles)
    const int i = i0 + grp;
    const bool ok = i <= depth && (!p.sc.window || i < p.sc.window || n + depth - i < p.sc.sink);
    const int64_t at = ok ? mine[i] : tok;
    Share<D> k, v;
    k.load(p.k, b * p.k.sb + at * p.k.st + (int64_t)h * p.k.sh, l8);
    v.load(p.v, b * p.v.sb + at * p.v.st + (int64_t)h * p.v.sh, l8);
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < Share<D>::kCh; ++e) dot = fmaf(q.v[e], k.v[e], dot);
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
    dot += __shfl_xor_sync(0xffffffffu, dot, 4);
    float x = dot * p.sc.factor;
    if (p.sc.cap2 > 0.0f) {
      float y = x;
      kv8_cap2(x, y, p.sc.cap2);
    }
    x = fmaf(-slope, (float)i, x);
    if (ok && x != -INFINITY) all.join(x, 1.0f, v.v);
  }

  // ---- the groups together
#pragma unroll
  for (int d = 8; d < 32; d *= 2) {
    float y[D / 8];
#pragma unroll
    for (int e = 0; e < D / 8; ++e) y[e] = __shfl_xor_sync(0xffffffffu, all.o[e], d);
    const float m = __shfl_xor_sync(0xffffffffu, all.top, d);
    const float s = __shfl_xor_sync(0xffffffffu, all.sum, d);
    all.join(m, s, y);
  }
  if (WARPS > 1) {
    if (lane < 8) {
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc)
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
    for (int w = 1; w < WARPS; ++w) {
      Share<D> y;
      y.load(outs[w], l8);
      all.join(stat[0][w], stat[1][w], y.v);
    }
  }
  if (lane < 8) {
    const float inv = all.sum == 0.0f ? 0.0f : 1.0f / all.sum;
    uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.a.out.data)) + b * p.a.out.sb +
                    (int64_t)tok * p.a.out.st + (int64_t)hd * p.a.out.sh;
#pragma unroll
    for (int cc = 0; cc < D / 64; ++cc) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack16(all.o[8 * cc + 2 * e] * inv, all.o[8 * cc + 2 * e + 1] * inv, p.a.out.type);
      *reinterpret_cast<uint4*>(out + 64 * cc + 8 * l8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (p.a.lse && lane == 0)
      p.a.lse[row] = all.sum == 0.0f ? -INFINITY : (all.top + log2f(all.sum)) * 0.6931471805599453f;
  }
}

template <int D>
cudaError_t join_as(const JoinParams& p, int num_sms, cudaStream_t s) {
  const int64_t rows = (int64_t)p.a.c.batch * p.a.T * p.a.H;
  // Few query rows: eight warps each, for the parts of a unit that many CTAs shared.
  if (rows <= 16 * num_sms)
    return kv8_launch(kv8_tree_join_kernel<D, kJoinWarps>, dim3((unsigned)rows), kJoinThreads, 0, s, p);
  return kv8_launch(kv8_tree_join_kernel<D, 1>, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)),
                    kJoinThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_kv8_tree_join(const Kv8Attn& a, const Kv8Scores& sc, const Kv8Left& left,
                                 const Kv8Rows& k, const Kv8Rows& v, int num_sms, cudaStream_t s) {
  const JoinParams p{a, sc, left, k, v};
  return a.D == 64 ? join_as<64>(p, num_sms, s) : join_as<128>(p, num_sms, s);
}

}  // namespace csa2
