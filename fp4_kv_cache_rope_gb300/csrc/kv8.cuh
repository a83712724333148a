// Shared pieces of the 8-bit K/V cache's kernels: the cache's addressing, the
// code formats, the scale rule and the split of the cached rows over CTAs.
//
// Storage: codes [pages, kv_heads, page rows, D] (a page's rows of one head are
// contiguous, so a tile of keys streams as one run), one fp32 scale per block
// of rows and head, always a power of two.  With a power of two the division
// x / s, the re-expression of a code under a larger scale and the product
// code * s are exact in fp32 but for the one rounding to the 8-bit format, so
// the stored bytes do not depend on how the arithmetic was arranged.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "codec.cuh"
#include "launch.h"

namespace csa2 {

constexpr int kKv8Ctas = 640;      // upper bound of the split kernels' CTAs
constexpr int kKv8SplitCtas = 256; // upper bound of the CTAs of a split prefill
constexpr int kKv8SlotRows = 24;   // query rows of one partial result
constexpr int kKv8Step = 128;      // cached rows of one step of a CTA

struct Kv8 {
  uint8_t* codes[2];               // K, V
  float* scales[2];
  float* mass;
  const int32_t* page_table;
  int32_t* seq_len;
  int32_t batch, heads, block_shift, page_rows, max_pages, max_len, num_pages, format;
  int32_t paged, page_shift;       // page_shift: log2(page_rows) or -1
};

// Column of the page table and row in the page of position t (contiguous: 0, t).
__device__ __forceinline__ int kv8_in_page(const Kv8& c, int t, int& in_page) {
  if (!c.paged) {
    in_page = t;
    return 0;
  }
  const uint32_t ut = (uint32_t)t;
  uint32_t pg;
  if (c.page_shift >= 0) {
    pg = ut >> c.page_shift;
    in_page = (int)(ut & (uint32_t)(c.page_rows - 1));
  } else {
    pg = ut / (uint32_t)c.page_rows;
    in_page = (int)(ut - pg * (uint32_t)c.page_rows);
  }
  return (int)pg;
}
// The page table's entry for position t, unchecked (contiguous: the sequence).
__device__ __forceinline__ int kv8_page_id(const Kv8& c, int b, int t) {
  int in_page;
  const int pg = kv8_in_page(c, t, in_page);
  return c.paged ? c.page_table[(int64_t)b * c.max_pages + pg] : b;
}
// The page, or -1 when its id is out of range.
__device__ __forceinline__ int kv8_check(const Kv8& c, int id) {
  return id < 0 || id >= c.num_pages ? -1 : id;
}
// Page (physical) and row in the page of position t of sequence b; page -1
// when the table's entry is out of range.
__device__ __forceinline__ int kv8_page(const Kv8& c, int b, int t, int& in_page) {
  const int pg = kv8_in_page(c, t, in_page);
  return kv8_check(c, c.paged ? c.page_table[(int64_t)b * c.max_pages + pg] : b);
}
// Row index over [pages, kv_heads, page rows]; times D for codes, as is for mass.
__device__ __forceinline__ int64_t kv8_row(const Kv8& c, int page, int h, int in_page) {
  return ((int64_t)page * c.heads + h) * c.page_rows + in_page;
}
// Index of the block's scale.
__device__ __forceinline__ int64_t kv8_block(const Kv8& c, int page, int h, int in_page) {
  return ((int64_t)page * c.heads + h) * (c.page_rows >> c.block_shift) + (in_page >> c.block_shift);
}
__device__ __forceinline__ int kv8_len(const Kv8& c, int b) {
  const int n = c.seq_len[b];
  return n < 0 ? 0 : (n > c.max_len ? c.max_len : n);
}

// ------------------------------------------------------------------- formats
// The smallest power of two s >= 2^-126 with amax <= qmax * s (qmax 448 = 1.75
// * 2^8, or 127 = 1.984375 * 2^6); 0 for amax = 0.  amax is finite.
template <int FMT>
__device__ __forceinline__ float kv8_scale_of(float amax) {
  if (amax == 0.0f) return 0.0f;
  const uint32_t u = __float_as_uint(amax);
  const int top = FMT == CSA2_KV8_E4M3 ? 8 : 6;
  const uint32_t lead = FMT == CSA2_KV8_E4M3 ? 0x600000u : 0x7E0000u;
  int e = (int)(u >> 23) - 127 - top + ((u & 0x7FFFFFu) > lead ? 1 : 0);
  e = e < -126 ? -126 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// 1/s of a power of two in [2^-126, 2^126]; 0 for 0.
__device__ __forceinline__ float kv8_inverse(float s) {
  return s == 0.0f ? 0.0f : __uint_as_float((254u << 23) - __float_as_uint(s));
}
// Four values already divided by the scale, finite and within +-qmax (the scale
// rule's promise), -> four codes: round to nearest, ties to even.  INT8: adding
// 1.5 * 2^23 rounds to an integer and leaves it in the low byte.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_encode4(float a, float b, float c, float d) {
  if (FMT == CSA2_KV8_E4M3) return e4m3x2_from_f32(a, b) | (e4m3x2_from_f32(c, d) << 16);
  const float k = 12582912.0f;
  const uint32_t lo = __byte_perm(__float_as_uint(a + k), __float_as_uint(b + k), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c + k), __float_as_uint(d + k), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
// Four codes -> two f16x2 (codes 0, 1 and 2, 3).  Exact.
template <int FMT>
__device__ __forceinline__ void kv8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == CSA2_KV8_E4M3) {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\n"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // v + 128 as the low byte of 1024 + (v + 128), then minus 1152
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
    __half2 hb = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<uint32_t*>(&ha);
    hi = *reinterpret_cast<uint32_t*>(&hb);
  }
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest magnitude among sixteen codes as a number that grows with it.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_max16(uint4 v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w}, even = 0, odd = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (FMT == CSA2_KV8_INT8) {
      const uint32_t neg = (w[i] >> 7) & 0x01010101u;          // |x|: ~x + 1 where negative
      w[i] = (w[i] ^ (neg * 255u)) + neg;                      // (-128 is no code)
    } else {
      w[i] &= 0x7F7F7F7Fu;
    }
    even = max_u16x2(even, w[i] & 0x00FF00FFu);
    odd = max_u16x2(odd, (w[i] >> 8) & 0x00FF00FFu);
  }
  const uint32_t m = max_u16x2(even, odd);
  return max(m & 0xFFFFu, m >> 16);
}
template <int FMT>
__device__ __forceinline__ float kv8_mag(uint32_t m) {
  return FMT == CSA2_KV8_E4M3 ? e4m3_decode(m) : (float)m;
}
// Four codes re-expressed times ratio (a power of two; the results lie within
// +-qmax), in f16: a code has at most 7 significant bits, so the product is
// exact wherever it does not round to 0 anyway (2^-24 against half of the
// smallest code, 2^-10 or 1/2), and is rounded to the format once.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_recode(uint32_t w, __half2 ratio) {
  uint32_t lo, hi;
  kv8_to_f16<FMT>(w, lo, hi);
  __half2 a = *reinterpret_cast<__half2*>(&lo), b = *reinterpret_cast<__half2*>(&hi);
  if (FMT == CSA2_KV8_E4M3) {
    a = __hmul2(a, ratio);
    b = __hmul2(b, ratio);
    uint32_t r;
    asm("{\n.reg .b16 x, y;\ncvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n"
        "cvt.rn.satfinite.e4m3x2.f16x2 y, %2;\nmov.b32 %0, {x, y};\n}"
        : "=r"(r)
        : "r"(*reinterpret_cast<uint32_t*>(&a)), "r"(*reinterpret_cast<uint32_t*>(&b)));
    return r;
  }
  // 1536 + v: v rounded to an integer, its low byte the code
  const __half2 k = __half2half2(__ushort_as_half((unsigned short)0x6600));
  a = __hfma2(a, ratio, k);
  b = __hfma2(b, ratio, k);
  return __byte_perm(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b), 0x6420);
}
// ratio as f16: below 2^-24 every product rounds to 0.
__device__ __forceinline__ __half2 kv8_ratio(float r) { return __float2half2_rn(r); }

// ------------------------------------------------------------------ row types
__device__ __forceinline__ void bf16x2_to_f32(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t pack16(float a, float b, int type) {
  if (type == CSA2_BF16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

__device__ __forceinline__ float kv8_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------- split of rows over the CTAs
// The steps (of kKv8Step cached rows) of all units are numbered through,
// sequence by sequence and within one unit by unit; CTA i of n takes the steps
// [W i / n, W (i+1) / n).  All sequences share the CTAs evenly whatever their
// lengths, which only the device knows.  Every sequence has at least one step.
__device__ __forceinline__ int kv8_steps(const Kv8& c, int b) {
  const int n = kv8_len(c, b);
  return n <= kKv8Step ? 1 : (n + kKv8Step - 1) / kKv8Step;
}
// Steps of one unit of all sequences (every lane of the warp gets it).
__device__ __forceinline__ int64_t kv8_total(const Kv8& c, int lane) {
  int64_t s = 0;
  for (int b = lane; b < c.batch; b += 32) s += kv8_steps(c, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
// CTAs that take part: each has a step at least, so that a unit's CTAs are
// consecutive and every partial result between them was written by this call.
__device__ __forceinline__ int kv8_sharers(int64_t total, int ctas) {
  return total < ctas ? (int)total : ctas;
}
// a * b / d (in 32 bits where they do: a 64-bit division is a long sequence)
__device__ __forceinline__ int64_t kv8_muldiv(int64_t a, int64_t b, int64_t d) {
  const int64_t y = a * b;
  if (y < (int64_t)1 << 32 && d < (int64_t)1 << 32) return (uint32_t)y / (uint32_t)d;
  return y / d;
}
// The sequence that holds step x when each has `units` units, and the step of
// its first unit (whole warp; x below the total).
__device__ __forceinline__ int kv8_find(const Kv8& c, int lane, int units, int64_t x,
                                        int64_t& first) {
  int64_t before = 0;
  for (int base = 0;; base += 32) {
    const int b = base + lane;
    const int64_t mine = b < c.batch ? (int64_t)kv8_steps(c, b) * units : 0;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > x);
    if (hit || base + 32 >= c.batch) {
      const int l = hit ? __ffs(hit) - 1 : 31;
      first = before + __shfl_sync(0xffffffffu, incl - mine, l);
      return min(base + l, c.batch - 1);
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// CTA `cta`'s first and last step, and where the first one lies.
struct Kv8Share {
  int ctas;               // CTAs that take part
  int64_t x, x1;          // steps [x, x1)
  int b, n, steps;        // the first step's sequence, its length and steps of a unit
  int unit, step;         // and the unit and its step
};
__device__ __forceinline__ Kv8Share kv8_share(const Kv8& c, int lane, int units, int max_ctas,
                                              int cta) {
  Kv8Share r;
  int64_t first;
  if (c.batch <= 32) {    // one look at the lengths
    const int n = lane < c.batch ? kv8_len(c, lane) : 0;
    const int mine = lane < c.batch ? (n <= kKv8Step ? 1 : (n + kKv8Step - 1) / kKv8Step) : 0;
    int incl = mine;      // at most 32 * 2^14 steps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int64_t total = (int64_t)__shfl_sync(0xffffffffu, incl, 31) * units;
    r.ctas = kv8_sharers(total, max_ctas);
    r.x = kv8_muldiv(total, cta, r.ctas);
    r.x1 = kv8_muldiv(total, cta + 1, r.ctas);
    const uint32_t hit = __ballot_sync(0xffffffffu, (int64_t)incl * units > r.x);
    r.b = hit ? __ffs(hit) - 1 : c.batch - 1;
    first = (int64_t)__shfl_sync(0xffffffffu, incl - mine, r.b) * units;
    r.n = __shfl_sync(0xffffffffu, n, r.b);
    r.steps = __shfl_sync(0xffffffffu, mine, r.b);
  } else {
    const int64_t total = kv8_total(c, lane) * units;
    r.ctas = kv8_sharers(total, max_ctas);
    r.x = kv8_muldiv(total, cta, r.ctas);
    r.x1 = kv8_muldiv(total, cta + 1, r.ctas);
    r.b = kv8_find(c, lane, units, r.x < total ? r.x : total - 1, first);
    r.n = kv8_len(c, r.b);
    r.steps = kv8_steps(c, r.b);
  }
  r.unit = (int)kv8_muldiv(r.x - first, 1, r.steps);
  r.step = (int)(r.x - first - (int64_t)r.unit * r.steps);
  return r;
}
// The CTAs c0 .. c1 that share unit `unit` of sequence b.
__device__ __forceinline__ void kv8_sharers_of(const Kv8& c, int lane, int units, int max_ctas,
                                               int b, int unit, int& c0, int& c1) {
  int64_t all = 0, before = 0;
  int steps = 0;
  for (int i = lane; i < c.batch; i += 32) {
    const int s = kv8_steps(c, i);
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
  // CTA i has the steps from total i / ctas on: step x is that of the last i
  // with total i < (x + 1) ctas
  c0 = (int)((((x0 + 1) * ctas - 1) < (int64_t)1 << 32 && total < (int64_t)1 << 32)
                 ? (uint32_t)((x0 + 1) * ctas - 1) / (uint32_t)total
                 : ((x0 + 1) * ctas - 1) / total);
  const int64_t e = (x0 + steps) * ctas - 1;
  c1 = (int)((e < (int64_t)1 << 32 && total < (int64_t)1 << 32) ? (uint32_t)e / (uint32_t)total
                                                                : e / total);
}

// ------------------------------------------------------------------ launchers
constexpr int kKv8Devices = 64;

// Gives the kernel `smem` dynamic bytes and the largest shared-memory carveout;
// the attributes stay with the device, so once per device and kernel (`seen` is
// the kernel's).  Setting them again, from another thread too, does no harm.
template <typename Kernel>
inline cudaError_t kv8_prepare(Kernel kern, int smem, std::atomic<uint64_t>& seen) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < kKv8Devices ? 1ull << dev : 0;
  if (seen.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = prefer_max_shared(kern);
  if (e == cudaSuccess) seen.fetch_or(bit, std::memory_order_relaxed);
  return e;
}
// One launch that may overlap the tail of the previous one of its stream.
template <typename... A>
inline cudaError_t kv8_launch(void (*kern)(A...), dim3 grid, int threads, size_t smem,
                              cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

struct Kv8Rows {          // rows [B, T, heads, D] with element strides
  const void* data;
  int64_t sb, st, sh;
  int32_t type;
};
struct Kv8Attn {
  Kv8 c;
  Kv8Rows q, out;         // out.data null: mass only
  float* lse;             // [B, T, H] or null (attention); read by mass
  const int32_t* q_len;   // [B] or null
  int32_t T, H, G, D;
  float scale_log2;       // softmax scale * log2(e), and
  float scale_low;        // what its rounding to fp32 left (mass)
  float decay;            // mass
  float* part;            // partial results
  uint32_t* status;
};
size_t kv8_part_bytes(int D);
size_t kv8_prefill_part_bytes(int D);
cudaError_t launch_kv8_prefill(const Kv8Attn& a, int num_sms, cudaStream_t s);
cudaError_t launch_kv8_append(const Kv8& c, int D, const Kv8Rows& k, const Kv8Rows& v, int T,
                              const int32_t* new_len, const int32_t* start, uint32_t* status,
                              cudaStream_t s);
cudaError_t launch_kv8_attn(const Kv8Attn& a, int num_sms, cudaStream_t s);
cudaError_t launch_kv8_mass_few(const Kv8Attn& a, int num_sms, cudaStream_t s);
cudaError_t launch_kv8_mass_many(const Kv8Attn& a, int num_sms, cudaStream_t s);
cudaError_t launch_kv8_evict(const Kv8& src, const Kv8& dst, bool in_place, int D, int keep,
                             int sink, int recent, int32_t* kept, int32_t* old_len,
                             uint32_t* status, int num_sms, cudaStream_t s);

}  // namespace csa2
