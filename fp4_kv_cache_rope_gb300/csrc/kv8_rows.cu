// The 8-bit K/V cache's append and eviction: rows into blocks of codes with
// one power-of-two scale per (block, head), and the rows that stay, moved into
// new blocks.  Both move bytes: their floor is the rows read once and written
// once.
#include "kv8.cuh"

namespace csa2 {
namespace {

struct AppendParams {
  Kv8 c;
  Kv8Rows in[2];           // K, V
  int32_t T;
  const int32_t* new_len;  // [B] or null (= T)
  const int32_t* start;    // [B] or null (= seq_len)
  uint32_t* status;
  int32_t own_len;         // the kernel itself writes seq_len
};

struct Span {
  int start, t;            // first position and number of the new rows (in range)
  bool over;
};
__device__ __forceinline__ Span append_span(const AppendParams& p, int b) {
  Span s;
  const int first = p.start ? p.start[b] : kv8_len(p.c, b);
  int t = p.new_len ? p.new_len[b] : p.T;
  t = t < 0 ? 0 : (t > p.T ? p.T : t);
  s.over = first < 0 || first > p.c.max_len || t > p.c.max_len - first;
  s.start = first < 0 ? 0 : (first > p.c.max_len ? p.c.max_len : first);
  if (first < 0) t = 0;
  s.t = t > p.c.max_len - s.start ? p.c.max_len - s.start : t;
  return s;
}

template <int NT>
__device__ __forceinline__ float group_max(float x, float* red, int tid) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if (NT == 32) {
    __syncwarp();
    return x;
  }
  __syncthreads();         // red may still be read from an earlier call
  if ((tid & 31) == 0) red[tid >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int i = 1; i < NT / 32; ++i) x = fmaxf(x, red[i]);
  return x;
}

// The new rows of one block, head and side (0 K, 1 V), by NT threads (a warp
// or a CTA).  The rows are held in registers between the block's maximum and
// their codes, so they are read once.
template <int D, int ES, int FMT, int NT, int PASSES>
__device__ __forceinline__ void append_block(const AppendParams& p, const Span& sp, int b, int h,
                                             int side, int blk, float* red, int tid) {
  constexpr int kLanes = D / 8;            // threads per row, 8 channels each
  constexpr int kRows = NT / kLanes;
  const Kv8& c = p.c;
  const int block = 1 << c.block_shift;
  const int b0 = blk << c.block_shift;
  const int lo = max(sp.start, b0), hi = min(sp.start + sp.t, b0 + block);
  if (lo >= hi) return;                    // uniform over the group
  int in_page;
  const int page = kv8_page(c, b, b0, in_page);
  if (page < 0) {
    if (tid == 0) set_status(p.status, CSA2_DEV_BAD_PAGE);
    return;
  }
  const Kv8Rows& in = p.in[side];
  const int sub = tid / kLanes, ch = (tid % kLanes) * 8;
  const char* src = static_cast<const char*>(in.data) +
                    (b * in.sb + (int64_t)(lo - sp.start) * in.st + h * in.sh + ch) * ES;
  const bool had = sp.start > b0;
  float* scale = c.scales[side] + kv8_block(c, page, h, in_page);
  const float s0 = had ? *scale : 0.0f;

  uint4 raw[PASSES][ES / 2];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * kRows + sub;
#pragma unroll
    for (int u = 0; u < ES / 2; ++u) {
      raw[i][u] = make_uint4(0, 0, 0, 0);
      if (lo + r < hi)
        raw[i][u] = reinterpret_cast<const uint4*>(src + (int64_t)r * in.st * ES)[u];
    }
  }
  auto values = [&](int i, float (&v)[8]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (ES == 4) {
        v[2 * j] = __uint_as_float(w[2 * j]);
        v[2 * j + 1] = __uint_as_float(w[2 * j + 1]);
      } else if (in.type == CSA2_BF16) {
        bf16x2_to_f32(w[j], v[2 * j], v[2 * j + 1]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  };
  float amax = 0.0f;
  bool odd = false;                        // an infinity or a NaN
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    float v[8];
    values(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(v[j]);
      const bool fin = a <= 3.402823466e38f;
      odd |= !fin;
      amax = fmaxf(amax, fin ? a : 0.0f);
    }
  }
  if (odd) set_status(p.status, CSA2_DEV_NONFINITE);
  amax = group_max<NT>(amax, red, tid);    // also: every thread has read s0
  const float s1 = fmaxf(s0, kv8_scale_of<FMT>(amax));
  const float inv = kv8_inverse(s1);
  const int64_t row0 = kv8_row(c, page, h, in_page);
  uint8_t* dst = c.codes[side] + (row0 + (lo - b0)) * D + ch;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * kRows + sub;
    if (lo + r >= hi) continue;
    float v[8];
    values(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] != v[j] ? 0.0f : v[j] * inv;
    if (odd) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] != v[j] ? 0.0f : v[j];   // inf * 0
    }
    uint2 w;
    w.x = kv8_encode4<FMT>(v[0], v[1], v[2], v[3]);
    w.y = kv8_encode4<FMT>(v[4], v[5], v[6], v[7]);
    *reinterpret_cast<uint2*>(dst + (int64_t)r * D) = w;
  }
  if (s1 > s0) {
    if (s0 > 0.0f) {                       // the block's earlier rows under the larger scale
      const float ratio = s0 * inv;
      uint8_t* old = c.codes[side] + row0 * D + ch;
      for (int r = sub; r < lo - b0; r += kRows) {
        uint2 w = *reinterpret_cast<uint2*>(old + (int64_t)r * D);
        w.x = kv8_recode<FMT>(w.x, ratio);
        w.y = kv8_recode<FMT>(w.y, ratio);
        *reinterpret_cast<uint2*>(old + (int64_t)r * D) = w;
      }
    }
  }
  if (tid == 0 && (s1 > s0 || !had)) *scale = s1;
  if (side == 0 && c.mass) {
    float* m = c.mass + row0 + (lo - b0);
    for (int r = tid; r < hi - lo; r += NT) m[r] = 0.0f;
  }
}

// Appends of a few rows: one CTA per sequence, a warp per (head, side), so that
// one launch also advances seq_len (every warp reads it before the barrier).
constexpr int kFewRows = 8;
template <int D, int ES, int FMT>
__global__ void __launch_bounds__(1024) kv8_append_few_kernel(AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const Span sp = append_span(p, b);
  __syncthreads();
  if (threadIdx.x == 0) {
    if (sp.over) set_status(p.status, CSA2_DEV_OVERFLOW);
    p.c.seq_len[b] = sp.start + sp.t;
  }
  if (sp.t == 0) return;
  const int first = sp.start >> p.c.block_shift, last = (sp.start + sp.t - 1) >> p.c.block_shift;
  for (int i = threadIdx.x >> 5; i < 2 * p.c.heads; i += warps)
    for (int blk = first; blk <= last; ++blk)
      append_block<D, ES, FMT, 32, kFewRows * D / 256>(p, sp, b, i >> 1, i & 1, blk, nullptr, lane);
}

// Longer appends: one CTA per (block, head, side, sequence).
constexpr int kAppendThreads = 256;
template <int D, int ES, int FMT>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(AppendParams p) {
  __shared__ float red[kAppendThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z;
  const Span sp = append_span(p, b);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (sp.over) set_status(p.status, CSA2_DEV_OVERFLOW);
    if (p.own_len) p.c.seq_len[b] = sp.start + sp.t;
  }
  if (sp.t == 0) return;
  append_block<D, ES, FMT, kAppendThreads, D / 16>(p, sp, b, blockIdx.y >> 1, blockIdx.y & 1,
                                                   (sp.start >> p.c.block_shift) + blockIdx.x, red,
                                                   threadIdx.x);
}
__global__ void kv8_advance_kernel(AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.c.batch) return;
  const Span sp = append_span(p, b);
  p.c.seq_len[b] = sp.start + sp.t;
}

template <int D, int ES, int FMT>
cudaError_t append_as(const AppendParams& p0, cudaStream_t s) {
  AppendParams p = p0;
  if (p.T <= kFewRows) {
    const int warps = 2 * p.c.heads < 32 ? 2 * p.c.heads : 32;
    return kv8_launch(kv8_append_few_kernel<D, ES, FMT>, dim3(p.c.batch), 32 * warps, 0, s, p);
  }
  const int block = 1 << p.c.block_shift;
  // with `start` given nothing in the launch reads seq_len, so it may write it
  p.own_len = p.start != nullptr;
  cudaError_t e = kv8_launch(kv8_append_kernel<D, ES, FMT>,
                         dim3((p.T + block - 2) / block + 1, 2 * p.c.heads, p.c.batch),
                         kAppendThreads, 0, s, p);
  if (e != cudaSuccess || p.own_len) return e;
  return kv8_launch(kv8_advance_kernel, dim3((p.c.batch + 127) / 128), 128, 0, s, p);
}
template <int D>
cudaError_t append_of(const AppendParams& p, cudaStream_t s) {
  const bool wide = p.in[0].type == CSA2_F32;
  if (p.c.format == CSA2_KV8_E4M3)
    return wide ? append_as<D, 4, CSA2_KV8_E4M3>(p, s) : append_as<D, 2, CSA2_KV8_E4M3>(p, s);
  return wide ? append_as<D, 4, CSA2_KV8_INT8>(p, s) : append_as<D, 2, CSA2_KV8_INT8>(p, s);
}

// ------------------------------------------------------------------- eviction
struct EvictParams {
  Kv8 src, dst;
  int32_t keep, sink, recent;
  int32_t* kept;       // [B, heads, keep]
  int32_t* old_len;    // [B]
  uint32_t* status;
  int32_t in_place;
};

// Larger weight -> larger key; both zeros alike, every NaN above all numbers.
__device__ __forceinline__ uint32_t rank_key(float x) {
  const uint32_t u = __float_as_uint(x), mag = u & 0x7FFFFFFFu;
  if (mag > 0x7F800000u) return 0xFFFFFFFFu;
  if (mag == 0) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Which rows stay, one CTA per (head, sequence): the threshold among the rows
// between the sink and the recent ones by a radix select over the order keys of
// their mass (8 bits a pass), then the kept rows in order by a running count.
constexpr int kSelThreads = 1024;
__global__ void __launch_bounds__(kSelThreads) kv8_evict_select_kernel(EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sh_prefix, sh_need;
  __shared__ int wsum[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const Kv8& c = p.src;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = kv8_len(c, b);
  if (h == 0 && tid == 0) p.old_len[b] = n;
  int32_t* kept = p.kept + ((int64_t)b * c.heads + h) * p.keep;
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int lo = p.sink, hi = n - p.recent;      // the ranked rows
  auto key_at = [&](int j) -> uint32_t {
    int in_page;
    const int page = kv8_page(c, b, j, in_page);
    if (page < 0) {
      set_status(p.status, CSA2_DEV_BAD_PAGE);
      return 0u;
    }
    return rank_key(c.mass[kv8_row(c, page, h, in_page)]);
  };
  if (tid == 0) {
    sh_prefix = 0;
    sh_need = (uint32_t)(p.keep - p.sink - p.recent);
  }
  __syncthreads();
  // after pass i: the top 8 (i+1) bits of the need-th largest key
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = sh_prefix;
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t k = key_at(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t need = sh_need;
      int d = 255;
      for (; d > 0 && hist[d] < need; --d) need -= hist[d];
      sh_prefix = prefix | ((uint32_t)d << shift);
      sh_need = need;                            // how many of the rows at the threshold stay
    }
    __syncthreads();
  }
  const uint32_t thr = sh_prefix;
  const uint32_t ties = p.keep - p.sink - p.recent == 0 ? 0u : sh_need;
  // in order: rows above the threshold, and the first `ties` rows at it
  int out = 0;
  uint32_t tied = 0;
  for (int base = 0; base < n; base += kSelThreads) {
    const int j = base + tid;
    bool always = j < n && (j < lo || j >= hi), above = false, at = false;
    if (j >= lo && j < hi && p.keep > p.sink + p.recent) {
      const uint32_t k = key_at(j);
      above = k > thr;
      at = k == thr;
    }
    const uint32_t bt = __ballot_sync(0xffffffffu, at);
    if (lane == 0) wsum[0][warp] = __popc(bt);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      before += w < warp ? wsum[0][w] : 0;
      all += wsum[0][w];
    }
    const uint32_t rank = tied + before + __popc(bt & ((1u << lane) - 1u));
    const bool keep = always || above || (at && rank < ties);
    tied += all;
    const uint32_t bk = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) wsum[1][warp] = __popc(bk);
    __syncthreads();
    before = 0;
    all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      before += w < warp ? wsum[1][w] : 0;
      all += wsum[1][w];
    }
    const int at_out = out + before + __popc(bk & ((1u << lane) - 1u));
    if (keep && at_out < p.keep) kept[at_out] = j;
    out += all;
  }
}

// One block of the result, by a CTA: the kept rows' codes in registers, their
// largest value, the new scale, the codes re-expressed.  Every read of the
// source comes before the first write.
constexpr int kMoveThreads = 256;
template <int D, int FMT>
__device__ void move_block(const EvictParams& p, int b, int h, int blk, int m, const int32_t* kept,
                           float* red) {
  constexpr int kLanes = D / 16;              // threads per row, 16 codes each
  constexpr int kRows = kMoveThreads / kLanes;
  constexpr int kPasses = 128 / kRows;
  const Kv8 &s = p.src, &d = p.dst;
  const int block = 1 << d.block_shift, b0 = blk << d.block_shift;
  const int rows = min(block, m - b0);
  const int tid = threadIdx.x, sub = tid / kLanes, ch = (tid % kLanes) * 16;
  int from[kPasses];
  bool moved = false;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + sub;
    from[i] = r < rows ? kept[b0 + r] : -1;
    moved |= r < rows && from[i] != b0 + r;
  }
  moved = __syncthreads_or(moved);
  if (p.in_place && !moved) return;
  int din;
  const int dpage = kv8_page(d, b, b0, din);
  if (dpage < 0 && tid == 0) set_status(p.status, CSA2_DEV_BAD_PAGE);
  const int64_t drow = kv8_row(d, dpage < 0 ? 0 : dpage, h, din);
  float mass[kPasses];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    uint4 code[kPasses];
    float scale[kPasses];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      code[i] = make_uint4(0, 0, 0, 0);
      scale[i] = 0.0f;
      if (side == 0) mass[i] = 0.0f;
      if (from[i] < 0) continue;
      int in_page;
      const int page = kv8_page(s, b, from[i], in_page);
      if (page < 0) {
        set_status(p.status, CSA2_DEV_BAD_PAGE);
        continue;
      }
      const int64_t row = kv8_row(s, page, h, in_page);
      code[i] = *reinterpret_cast<const uint4*>(s.codes[side] + row * D + ch);
      scale[i] = s.scales[side][kv8_block(s, page, h, in_page)];
      if (side == 0 && s.mass) mass[i] = s.mass[row];
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t mx = max(max(kv8_max4<FMT>(code[i].x), kv8_max4<FMT>(code[i].y)),
                              max(kv8_max4<FMT>(code[i].z), kv8_max4<FMT>(code[i].w)));
      amax = fmaxf(amax, kv8_mag<FMT>(mx) * scale[i]);
    }
    amax = group_max<kMoveThreads>(amax, red, tid);   // every read is behind this
    const float s1 = kv8_scale_of<FMT>(amax);
    const float inv = kv8_inverse(s1);
    if (dpage < 0) continue;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRows + sub;
      if (r >= rows) continue;
      uint4 w = code[i];
      const float ratio = scale[i] * inv;
      if (moved && ratio != 1.0f) {
        w.x = kv8_recode<FMT>(w.x, ratio);
        w.y = kv8_recode<FMT>(w.y, ratio);
        w.z = kv8_recode<FMT>(w.z, ratio);
        w.w = kv8_recode<FMT>(w.w, ratio);
      }
      *reinterpret_cast<uint4*>(d.codes[side] + (drow + r) * D + ch) = w;
      if (side == 0 && ch == 0 && d.mass) d.mass[drow + r] = mass[i];
      if (r == 0 && ch == 0) d.scales[side][kv8_block(d, dpage, h, din)] = moved ? s1 : scale[i];
    }
  }
}

// Into another cache: one CTA per (block, head, sequence).  In place: one CTA
// per (head, sequence) walks the blocks upwards.  A kept row never moves to a
// later place, so the sources of the blocks still to come lie behind the block
// being written.
template <int D, int FMT>
__global__ void __launch_bounds__(kMoveThreads) kv8_evict_move_kernel(EvictParams p) {
  __shared__ float red[kMoveThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.y, b = blockIdx.z;
  const int n = p.old_len[b], m = min(n, p.keep);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.dst.seq_len[b] = m;
  if (p.in_place && n == m) return;
  const int32_t* kept = p.kept + ((int64_t)b * p.src.heads + h) * p.keep;
  const int blocks = (m + (1 << p.dst.block_shift) - 1) >> p.dst.block_shift;
  for (int blk = blockIdx.x; blk < blocks; blk += gridDim.x)
    move_block<D, FMT>(p, b, h, blk, m, kept, red);
}

template <int D, int FMT>
cudaError_t move_as(const EvictParams& p, cudaStream_t s) {
  const int blocks = (p.keep + (1 << p.dst.block_shift) - 1) >> p.dst.block_shift;
  return kv8_launch(kv8_evict_move_kernel<D, FMT>,
                dim3(p.in_place ? 1 : blocks, p.src.heads, p.src.batch), kMoveThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8& c, int D, const Kv8Rows& k, const Kv8Rows& v, int T,
                              const int32_t* new_len, const int32_t* start, uint32_t* status,
                              cudaStream_t s) {
  AppendParams p{c, {k, v}, T, new_len, start, status, 0};
  return D == 64 ? append_of<64>(p, s) : append_of<128>(p, s);
}

cudaError_t launch_kv8_evict(const Kv8& src, const Kv8& dst, bool in_place, int D, int keep,
                             int sink, int recent, int32_t* kept, int32_t* old_len,
                             uint32_t* status, int num_sms, cudaStream_t s) {
  EvictParams p{src, dst, keep, sink, recent, kept, old_len, status, in_place ? 1 : 0};
  cudaError_t e = kv8_launch(kv8_evict_select_kernel, dim3(src.heads, src.batch), kSelThreads, 0,
                         s, p);
  if (e != cudaSuccess) return e;
  if (src.format == CSA2_KV8_E4M3)
    return D == 64 ? move_as<64, CSA2_KV8_E4M3>(p, s) : move_as<128, CSA2_KV8_E4M3>(p, s);
  return D == 64 ? move_as<64, CSA2_KV8_INT8>(p, s) : move_as<128, CSA2_KV8_INT8>(p, s);
}

}  // namespace csa2
