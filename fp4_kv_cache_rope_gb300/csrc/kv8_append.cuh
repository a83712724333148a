// Rows into blocks of codes with one power-of-two scale per (block, head): the
// 8-bit cache's append.  It moves bytes: its floor is the rows read once and
// written once.
#pragma once

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
  const int32_t* path;     // [B, T]: rows of `in` that are appended, or null (all in order)
  int32_t in_rows;         // rows of a sequence in `in` (path only)
};

struct Span {
  int start, t;            // first position and number of the new rows (in range)
  int first, given;        // as they were given (the number within 0 .. T)
  bool over;
};
__device__ __forceinline__ Span append_span(const AppendParams& p, int b) {
  Span s;
  const int first = p.start ? p.start[b] : kv8_len(p.c, b);
  int t = p.new_len ? p.new_len[b] : p.T;
  t = t < 0 ? 0 : (t > p.T ? p.T : t);
  s.first = min(first, 1 << 30);
  s.given = t;
  s.over = first < 0 || first > p.c.max_len || t > p.c.max_len - first;
  s.start = first < 0 ? 0 : (first > p.c.max_len ? p.c.max_len : first);
  if (first < 0) t = 0;
  s.t = t > p.c.max_len - s.start ? p.c.max_len - s.start : t;
  return s;
}

// Largest of the NT threads' values (a warp's or a CTA's).
template <int NT>
__device__ __forceinline__ uint32_t group_max(uint32_t x, uint32_t* red, int tid) {
  x = __reduce_max_sync(0xffffffffu, x);
  if (NT == 32) return x;
  __syncthreads();         // red may still be read from an earlier call
  if ((tid & 31) == 0) red[tid >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int i = 1; i < NT / 32; ++i) x = max(x, red[i]);
  return x;
}

// A block's scale raised from s0 to s1 = 1 / inv: its n earlier rows (from row0 on) under the
// larger one.
template <int D, int FMT, int NT>
__device__ __forceinline__ void block_rescale(uint8_t* codes, float* scale, float s0, float s1,
                                              float inv, int64_t row0, int n, int tid) {
  if (s1 > s0 && s0 > 0.0f) {
    const __half2 ratio = kv8_ratio(s0 * inv);
    uint8_t* old = codes + row0 * D;
    for (int i = tid; i < n * D / 8; i += NT) {
      uint2 w = *reinterpret_cast<uint2*>(old + 8 * i);
      w.x = kv8_recode<FMT>(w.x, ratio);
      w.y = kv8_recode<FMT>(w.y, ratio);
      *reinterpret_cast<uint2*>(old + 8 * i) = w;
    }
  }
  if (tid == 0 && (s1 > s0 || n == 0)) *scale = s1;
}

// The new rows of one block and head, K and V, by NT threads (a warp or a CTA),
// 16 bytes a thread and access.  The rows are held in registers between the
// block's maximum and their codes, so they are read once; where the registers
// allow it both sides are read before either is worked on.  The maximum is taken
// over the bits of the magnitudes (two 16-bit values at a time), which also
// shows whether there is an infinity or a NaN.
// TYPE: the rows' type.  PATH: the rows are chosen by p.path.
template <int D, int TYPE, int NT, int PASSES, bool PATH = false>
struct NewRows {
  static constexpr int EL = TYPE == CSA2_F32 ? 4 : 8;   // elements per 16 bytes
  static constexpr int kLanes = D / EL;                 // threads per row
  static constexpr int kRows = NT / kLanes;
  static constexpr uint32_t kInf = TYPE == CSA2_F32 ? 0x7F800000u : TYPE == CSA2_BF16 ? 0x7F80u : 0x7C00u;
  uint4 raw[PASSES];
  float s0;                                // the block's scale so far

  __device__ __forceinline__ void read(const AppendParams& p, const Kv8Rows& in, const Span& sp,
                                       int b, int h, int lo, int hi, bool had, const float* scale,
                                       int tid) {
    const int sub = tid / kLanes, ch = (tid % kLanes) * EL;
    if (PATH) {
      const char* src = static_cast<const char*>(in.data) + (b * in.sb + h * in.sh + ch) * (16 / EL);
      const int32_t* path = p.path + (int64_t)b * p.T + (lo - sp.start + sub);
      s0 = had ? *scale : 0.0f;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        raw[i] = make_uint4(0, 0, 0, 0);
        if (lo + i * kRows + sub >= hi) continue;
        const int at = path[i * kRows];
        if (at >= 0 && at < p.in_rows)
          raw[i] = *reinterpret_cast<const uint4*>(src + (int64_t)at * in.st * (16 / EL));
        else
          set_status(p.status, CSA2_DEV_BAD_INDEX);
      }
      return;
    }
    const char* src = static_cast<const char*>(in.data) +
                      (b * in.sb + (int64_t)(lo - sp.start + sub) * in.st + h * in.sh + ch) * (16 / EL);
    const int64_t step = (int64_t)kRows * in.st * (16 / EL);
    s0 = had ? *scale : 0.0f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (lo + i * kRows + sub < hi) raw[i] = *reinterpret_cast<const uint4*>(src + i * step);
    }
  }

  // the elements of word j of an access, times inv (a power of two)
  static __device__ __forceinline__ void scaled(uint32_t w, float inv, float (&v)[2]) {
    if (TYPE == CSA2_F32) {
      v[0] = __uint_as_float(w) * inv;
    } else if (TYPE == CSA2_BF16) {
      // exact in bf16 too, whose exponents are fp32's
      const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w),
                                       __float2bfloat162_rn(inv));
      bf16x2_to_f32(*reinterpret_cast<const uint32_t*>(&x), v[0], v[1]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
      v[0] = f.x * inv;
      v[1] = f.y * inv;
    }
  }

  // row0: index of the block's first row; lo, hi: the new rows' positions
  template <int FMT>
  __device__ __forceinline__ void write(const AppendParams& p, uint8_t* codes, float* scale,
                                        int64_t row0, int b0, int lo, int hi, uint32_t* red, int tid) {
    const int sub = tid / kLanes, ch = (tid % kLanes) * EL;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        bits = EL == 4 ? max(bits, w[j] & 0x7FFFFFFFu) : max_u16x2(bits, w[j] & 0x7FFF7FFFu);
    }
    if (EL == 8) bits = max(bits & 0xFFFFu, bits >> 16);
    bits = group_max<NT>(bits, red, tid);
    const bool odd = bits >= kInf;         // uniform over the group
    if (odd) {                             // the maximum of the finite values then
      if (tid == 0) set_status(p.status, CSA2_DEV_NONFINITE);
      bits = 0;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < EL / 4; ++e) {
            const uint32_t m = EL == 4 ? w[j] & 0x7FFFFFFFu : (w[j] >> (16 * e)) & 0x7FFFu;
            if (m < kInf) bits = max(bits, m);
          }
      }
      bits = group_max<NT>(bits, red, tid);
    }
    __syncwarp();                          // every thread of the group has read s0
    const float amax = TYPE == CSA2_F32 ? __uint_as_float(bits)
                       : TYPE == CSA2_BF16
                           ? __uint_as_float(bits << 16)
                           : __half2float(__ushort_as_half((unsigned short)bits));
    const float s1 = fmaxf(s0, kv8_scale_of<FMT>(amax));
    const float inv = kv8_inverse(s1);
    uint8_t* dst = codes + (row0 + (lo - b0) + sub) * D + ch;
    if (odd) {                             // infinities and NaN among the rows
      const float big = s1 > 0.0f ? (FMT == CSA2_KV8_E4M3 ? 448.0f : 127.0f) : 0.0f;
#pragma unroll 1
      for (int i = 0; i < PASSES; ++i) {
        if (lo + i * kRows + sub >= hi) continue;
        uint4 r = raw[0];
#pragma unroll
        for (int k = 1; k < PASSES; ++k)
          if (k == i) r = raw[k];
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x[2];
          scaled(w[j], 1.0f, x);
          if (EL == 4) v[j] = x[0];
          else v[2 * j] = x[0], v[2 * j + 1] = x[1];
        }
#pragma unroll
        for (int j = 0; j < EL; ++j)
          v[j] = fabsf(v[j]) <= 3.402823466e38f ? v[j] * inv : v[j] != v[j] ? 0.0f : copysignf(big, v[j]);
        store<FMT>(dst + (int64_t)i * kRows * D, v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        if (lo + i * kRows + sub >= hi) continue;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x[2];
          scaled(w[j], inv, x);
          if (EL == 4) v[j] = x[0];
          else v[2 * j] = x[0], v[2 * j + 1] = x[1];
        }
        store<FMT>(dst + (int64_t)i * kRows * D, v);
      }
    }
    block_rescale<D, FMT, NT>(codes, scale, s0, s1, inv, row0, lo - b0, tid);
  }

  template <int FMT>
  static __device__ __forceinline__ void store(uint8_t* to, const float (&v)[8]) {
    if (EL == 4)
      *reinterpret_cast<uint32_t*>(to) = kv8_encode4<FMT>(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(kv8_encode4<FMT>(v[0], v[1], v[2], v[3]),
                                                 kv8_encode4<FMT>(v[4], v[5], v[6], v[7]));
  }
};

template <int D, int TYPE, int FMT, int NT, int PASSES, int SIDES, bool PATH>
__device__ __forceinline__ void append_block(const AppendParams& p, const Span& sp, int b, int h,
                                             int side, int blk, uint32_t* red, int tid) {
  const Kv8& c = p.c;
  const int b0 = blk << c.block_shift;
  const int lo = max(sp.start, b0), hi = min(sp.start + sp.t, b0 + (1 << c.block_shift));
  if (lo >= hi) return;                    // uniform over the group
  int in_page;
  const int page = kv8_page(c, b, b0, in_page);
  if (page < 0) {
    if (tid == 0) set_status(p.status, CSA2_DEV_BAD_PAGE);
    return;
  }
  const int64_t row0 = kv8_row(c, page, h, in_page), at = kv8_block(c, page, h, in_page);
  const bool had = sp.start > b0;
  if (SIDES == 2) {
    NewRows<D, TYPE, NT, PASSES, PATH> k, v;
    k.read(p, p.in[0], sp, b, h, lo, hi, had, c.scales[0] + at, tid);
    v.read(p, p.in[1], sp, b, h, lo, hi, had, c.scales[1] + at, tid);
    k.template write<FMT>(p, c.codes[0], c.scales[0] + at, row0, b0, lo, hi, red, tid);
    v.template write<FMT>(p, c.codes[1], c.scales[1] + at, row0, b0, lo, hi, red, tid);
  } else {
    NewRows<D, TYPE, NT, PASSES, PATH> x;
    x.read(p, p.in[side], sp, b, h, lo, hi, had, c.scales[side] + at, tid);
    x.template write<FMT>(p, c.codes[side], c.scales[side] + at, row0, b0, lo, hi, red, tid);
  }
  if (side == 0 && c.mass)
    for (int r = tid; r < hi - lo; r += NT) c.mass[row0 + (lo - b0) + r] = 0.0f;
}

// Appends of a few rows: one CTA per sequence, a warp per (head, side), so that
// one launch also advances seq_len (every warp reads it before the barrier).
// Latency: one token of 32 sequences takes 5 us, and 0.1 MB moves.
constexpr int kFewRows = 8;
template <int D, int TYPE, int FMT, bool PATH>
__global__ void __launch_bounds__(512) kv8_append_few_kernel(AppendParams p) {
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
      append_block<D, TYPE, FMT, 32, kFewRows * D / NewRows<D, TYPE, 32, 1>::EL / 32, 1, PATH>(
          p, sp, b, i >> 1, i & 1, blk, nullptr, lane);
}

// Longer appends: one CTA per (block, head, sequence), or side of it.  PASSES:
// 16-byte accesses of a thread that hold a side of a block.  Bound by HBM: four
// prompts of 1280 to 8192 rows, 8 heads, D 128, bf16: 145 MB in 26 us, 5.5 TB/s.
constexpr int kAppendThreads = 256;
constexpr int append_sides(int passes) { return passes <= 8 ? 2 : 1; }
template <int D, int TYPE, int FMT, int PASSES, bool PATH>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(AppendParams p) {
  __shared__ uint32_t red[kAppendThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z;
  const Span sp = append_span(p, b);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (sp.over) set_status(p.status, CSA2_DEV_OVERFLOW);
    if (p.own_len) p.c.seq_len[b] = sp.start + sp.t;
  }
  if (sp.t == 0) return;
  constexpr int kSides = append_sides(PASSES);
  append_block<D, TYPE, FMT, kAppendThreads, PASSES, kSides, PATH>(
      p, sp, b, kSides == 2 ? blockIdx.y : blockIdx.y >> 1, kSides == 2 ? 0 : blockIdx.y & 1,
      (sp.start >> p.c.block_shift) + blockIdx.x, red, threadIdx.x);
}
__global__ void kv8_advance_kernel(AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.c.batch) return;
  const Span sp = append_span(p, b);
  p.c.seq_len[b] = sp.start + sp.t;
}

template <int D, int TYPE, int FMT, bool PATH>
cudaError_t append_as(const AppendParams& p0, cudaStream_t s) {
  AppendParams p = p0;
  if (p.T <= kFewRows) {
    const int warps = 2 * p.c.heads < 16 ? 2 * p.c.heads : 16;
    return kv8_launch(kv8_append_few_kernel<D, TYPE, FMT, PATH>, dim3(p.c.batch), 32 * warps, 0, s, p);
  }
  const int block = 1 << p.c.block_shift;
  // with `start` given nothing in the launch reads seq_len, so it may write it
  // (`start` may be seq_len itself)
  p.own_len = p.start != nullptr && p.start != p.c.seq_len;
  auto run = [&](auto kern, int passes) {
    const dim3 grid((p.T + block - 2) / block + 1, p.c.heads * (append_sides(passes) == 2 ? 1 : 2),
                    p.c.batch);
    return kv8_launch(kern, grid, kAppendThreads, 0, s, p);
  };
  constexpr int kMost = 128 * D / (TYPE == CSA2_F32 ? 4 : 8) / kAppendThreads;   // passes of 128 rows
  const cudaError_t e = block == 128 ? run(kv8_append_kernel<D, TYPE, FMT, kMost, PATH>, kMost)
                        : block == 64 ? run(kv8_append_kernel<D, TYPE, FMT, kMost / 2, PATH>, kMost / 2)
                                      : run(kv8_append_kernel<D, TYPE, FMT, kMost / 4, PATH>, kMost / 4);
  if (e != cudaSuccess || p.own_len) return e;
  return kv8_launch(kv8_advance_kernel, dim3((p.c.batch + 127) / 128), 128, 0, s, p);
}
template <int D, int FMT, bool PATH>
cudaError_t append_of(const AppendParams& p, cudaStream_t s) {
  return p.in[0].type == CSA2_F32    ? append_as<D, CSA2_F32, FMT, PATH>(p, s)
         : p.in[0].type == CSA2_BF16 ? append_as<D, CSA2_BF16, FMT, PATH>(p, s)
                                     : append_as<D, CSA2_F16, FMT, PATH>(p, s);
}
template <bool PATH>
cudaError_t append_any(const AppendParams& p, int D, cudaStream_t s) {
  if (p.c.format == CSA2_KV8_E4M3)
    return D == 64 ? append_of<64, CSA2_KV8_E4M3, PATH>(p, s) : append_of<128, CSA2_KV8_E4M3, PATH>(p, s);
  return D == 64 ? append_of<64, CSA2_KV8_INT8, PATH>(p, s) : append_of<128, CSA2_KV8_INT8, PATH>(p, s);
}

}  // namespace
}  // namespace csa2
