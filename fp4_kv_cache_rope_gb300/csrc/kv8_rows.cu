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

// The new rows of one block and head, K and V, by NT threads (a warp or a CTA),
// 16 bytes a thread and access.  The rows are held in registers between the
// block's maximum and their codes, so they are read once; where the registers
// allow it both sides are read before either is worked on.  The maximum is taken
// over the bits of the magnitudes (two 16-bit values at a time), which also
// shows whether there is an infinity or a NaN.
// TYPE: the rows' type.
template <int D, int TYPE, int NT, int PASSES>
struct NewRows {
  static constexpr int EL = TYPE == CSA2_F32 ? 4 : 8;   // elements per 16 bytes
  static constexpr int kLanes = D / EL;                 // threads per row
  static constexpr int kRows = NT / kLanes;
  static constexpr uint32_t kInf = TYPE == CSA2_F32 ? 0x7F800000u : TYPE == CSA2_BF16 ? 0x7F80u : 0x7C00u;
  uint4 raw[PASSES];
  float s0;                                // the block's scale so far

  __device__ __forceinline__ void read(const Kv8Rows& in, const Span& sp, int b, int h, int lo,
                                       int hi, bool had, const float* scale, int tid) {
    const int sub = tid / kLanes, ch = (tid % kLanes) * EL;
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
    if (s1 > s0 && s0 > 0.0f) {            // the block's earlier rows under the larger scale
      const __half2 ratio = kv8_ratio(s0 * inv);
      uint8_t* old = codes + row0 * D;
      for (int i = tid; i < (lo - b0) * D / 8; i += NT) {
        uint2 w = *reinterpret_cast<uint2*>(old + 8 * i);
        w.x = kv8_recode<FMT>(w.x, ratio);
        w.y = kv8_recode<FMT>(w.y, ratio);
        *reinterpret_cast<uint2*>(old + 8 * i) = w;
      }
    }
    if (tid == 0 && (s1 > s0 || lo == b0)) *scale = s1;
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

template <int D, int TYPE, int FMT, int NT, int PASSES, int SIDES>
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
    NewRows<D, TYPE, NT, PASSES> k, v;
    k.read(p.in[0], sp, b, h, lo, hi, had, c.scales[0] + at, tid);
    v.read(p.in[1], sp, b, h, lo, hi, had, c.scales[1] + at, tid);
    k.template write<FMT>(p, c.codes[0], c.scales[0] + at, row0, b0, lo, hi, red, tid);
    v.template write<FMT>(p, c.codes[1], c.scales[1] + at, row0, b0, lo, hi, red, tid);
  } else {
    NewRows<D, TYPE, NT, PASSES> x;
    x.read(p.in[side], sp, b, h, lo, hi, had, c.scales[side] + at, tid);
    x.template write<FMT>(p, c.codes[side], c.scales[side] + at, row0, b0, lo, hi, red, tid);
  }
  if (side == 0 && c.mass)
    for (int r = tid; r < hi - lo; r += NT) c.mass[row0 + (lo - b0) + r] = 0.0f;
}

// Appends of a few rows: one CTA per sequence, a warp per (head, side), so that
// one launch also advances seq_len (every warp reads it before the barrier).
// Latency: one token of 32 sequences takes 5 us, and 0.1 MB moves.
constexpr int kFewRows = 8;
template <int D, int TYPE, int FMT>
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
      append_block<D, TYPE, FMT, 32, kFewRows * D / NewRows<D, TYPE, 32, 1>::EL / 32, 1>(
          p, sp, b, i >> 1, i & 1, blk, nullptr, lane);
}

// Longer appends: one CTA per (block, head, sequence), or side of it.  PASSES:
// 16-byte accesses of a thread that hold a side of a block.  Bound by HBM: four
// prompts of 1280 to 8192 rows, 8 heads, D 128, bf16: 145 MB in 26 us, 5.5 TB/s.
constexpr int kAppendThreads = 256;
constexpr int append_sides(int passes) { return passes <= 8 ? 2 : 1; }
template <int D, int TYPE, int FMT, int PASSES>
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
  append_block<D, TYPE, FMT, kAppendThreads, PASSES, kSides>(
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

template <int D, int TYPE, int FMT>
cudaError_t append_as(const AppendParams& p0, cudaStream_t s) {
  AppendParams p = p0;
  if (p.T <= kFewRows) {
    const int warps = 2 * p.c.heads < 16 ? 2 * p.c.heads : 16;
    return kv8_launch(kv8_append_few_kernel<D, TYPE, FMT>, dim3(p.c.batch), 32 * warps, 0, s, p);
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
  const cudaError_t e = block == 128 ? run(kv8_append_kernel<D, TYPE, FMT, kMost>, kMost)
                        : block == 64 ? run(kv8_append_kernel<D, TYPE, FMT, kMost / 2>, kMost / 2)
                                      : run(kv8_append_kernel<D, TYPE, FMT, kMost / 4>, kMost / 4);
  if (e != cudaSuccess || p.own_len) return e;
  return kv8_launch(kv8_advance_kernel, dim3((p.c.batch + 127) / 128), 128, 0, s, p);
}
template <int D, int FMT>
cudaError_t append_of(const AppendParams& p, cudaStream_t s) {
  return p.in[0].type == CSA2_F32    ? append_as<D, CSA2_F32, FMT>(p, s)
         : p.in[0].type == CSA2_BF16 ? append_as<D, CSA2_BF16, FMT>(p, s)
                                     : append_as<D, CSA2_F16, FMT>(p, s);
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

// Which rows stay.  A cluster of CTAs per (head, sequence); each warp has a run
// of consecutive rows.  The need-th largest key is found 8 bits a pass: every
// CTA counts its rows' digits, the counts are added up over the cluster, and all
// CTAs walk the sum alike.  Rows above that key stay, and of those at it the
// first ones in order; both are counted per warp first, so that every warp knows
// its rows' places in `kept`.  Bound by latency (one round of the cluster's
// barrier per pass), not by the 4 bytes per row that it reads: 18 us for 4
// sequences of up to 32768 rows and 8 heads, 11 us for one of 1100.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelHeld = 16;       // keys that a thread keeps in registers
__global__ void __launch_bounds__(kSelThreads) kv8_evict_select_kernel(EvictParams p) {
  __shared__ uint32_t hist[2][256];                // this CTA's counts, by pass parity
  __shared__ uint32_t sum[256];
  __shared__ uint32_t sh_digit, sh_need;
  __shared__ int cnt[2][kSelWarps];                // rows above / at the threshold, per warp
  __shared__ int total[2];
  const Kv8& c = p.src;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank(), size = cluster_size();
  griddep_wait();
  griddep_launch_dependents();
  const int n = kv8_len(c, b);
  if (h == 0 && rank == 0 && tid == 0) p.old_len[b] = n;
  int32_t* kept = p.kept + ((int64_t)b * c.heads + h) * p.keep;
  if (n <= p.keep) {                               // uniform over the cluster
    for (int i = rank * kSelThreads + tid; i < p.keep; i += size * kSelThreads)
      kept[i] = i < n ? i : -1;
    return;
  }
  const int lo = p.sink, hi = n - p.recent;        // the ranked rows
  const int per = (n + size * kSelWarps * 32 - 1) / (size * kSelWarps * 32);   // rows a thread
  const int row0 = (rank * kSelWarps + warp) * per * 32 + lane;
  auto key_at = [&](int j) -> uint32_t {
    int in_page;
    const int page = kv8_page(c, b, j, in_page);
    if (page < 0) {
      set_status(p.status, CSA2_DEV_BAD_PAGE);
      return 0u;
    }
    return rank_key(c.mass[kv8_row(c, page, h, in_page)]);
  };
  uint32_t held[kSelHeld];
#pragma unroll
  for (int e = 0; e < kSelHeld; ++e) {
    const int j = row0 + 32 * e;
    held[e] = 0;
    if (e < per && j >= lo && j < hi) held[e] = key_at(j);
  }
  // f(row, key) for each ranked row of the thread, in order
  auto each = [&](auto f) {
#pragma unroll
    for (int e = 0; e < kSelHeld; ++e) {
      const int j = row0 + 32 * e;
      if (e < per) f(j, j >= lo && j < hi, held[e]);
    }
    for (int e = kSelHeld; e < per; ++e) {
      const int j = row0 + 32 * e;
      const bool in = j >= lo && j < hi;
      f(j, in, in ? key_at(j) : 0u);
    }
  };
  uint32_t prefix = 0;
  uint32_t need = (uint32_t)(p.keep - p.sink - p.recent);
  const bool any = need > 0;
  for (int shift = 24; any && shift >= 0; shift -= 8) {
    uint32_t* mine = hist[(shift >> 3) & 1];
    if (tid < 256) mine[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    each([&](int, bool in, uint32_t k) {
      const bool hit = in && (k & mask) == prefix;
      const uint32_t d = hit ? (k >> shift) & 255u : 256u;
      if (shift == 24) {     // weights share their leading bits: equal digits add once
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        if (hit && lane == __ffs(same) - 1) atomicAdd(&mine[d], (uint32_t)__popc(same));
      } else if (hit) {
        atomicAdd(&mine[d], 1u);
      }
    });
    cluster_sync();
    if (tid < 256) {
      uint32_t s = 0;
      for (int r = 0; r < size; ++r) s += peer_u32(&mine[tid], r);
      sum[tid] = s;
    }
    __syncthreads();
    if (warp == 0) {
      // lane l: digits 255 - 8 l downwards; how many rows lie above them
      uint32_t own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) own += sum[255 - 8 * lane - i];
      uint32_t above = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += y;
      }
      above -= own;
      if (above < need && above + own >= need) {
        uint32_t left = need - above;
        int d = 255 - 8 * lane;
        for (; sum[d] < left; --d) left -= sum[d];
        sh_digit = (uint32_t)d;
        sh_need = left;
      }
    }
    __syncthreads();
    prefix |= sh_digit << shift;
    need = sh_need;                                // rows at the threshold that stay
  }
  // ---- counts per warp, then the number of kept rows in front of it
  int above = 0, at = 0;
  each([&](int j, bool in, uint32_t k) {
    const bool up = j < n && (!in || (any && k > prefix));
    above += __popc(__ballot_sync(0xffffffffu, up));
    at += __popc(__ballot_sync(0xffffffffu, in && any && k == prefix));
  });
  if (lane == 0) {
    cnt[0][warp] = above;
    cnt[1][warp] = at;
  }
  __syncthreads();
  if (tid < 2) {
    int t = 0;
    for (int w = 0; w < kSelWarps; ++w) t += cnt[tid][w];
    total[tid] = t;
  }
  cluster_sync();
  int before_up = 0, before_at = 0;
  for (int r = 0; r < rank; ++r) {
    before_up += (int)peer_u32(&total[0], r);
    before_at += (int)peer_u32(&total[1], r);
  }
  for (int w = 0; w < warp; ++w) {
    before_up += cnt[0][w];
    before_at += cnt[1][w];
  }
  const uint32_t under = (1u << lane) - 1u;
  each([&](int j, bool in, uint32_t k) {
    const bool up = j < n && (!in || (any && k > prefix)), eq = in && any && k == prefix;
    const uint32_t bu = __ballot_sync(0xffffffffu, up), be = __ballot_sync(0xffffffffu, eq);
    const int r = before_at + __popc(be & under);  // place among the rows at the threshold
    const bool stay = up || (eq && r < (int)need);
    const int to = before_up + __popc(bu & under) + min(r, (int)need);
    if (stay && to < p.keep) kept[to] = j;
    before_up += __popc(bu);
    before_at += __popc(be);
  });
  cluster_sync();                                  // peers may still read this CTA's counts
}

template <int FMT>
__device__ __forceinline__ uint4 recode16(uint4 w, __half2 ratio) {
  return make_uint4(kv8_recode<FMT>(w.x, ratio), kv8_recode<FMT>(w.y, ratio),
                    kv8_recode<FMT>(w.z, ratio), kv8_recode<FMT>(w.w, ratio));
}

// A block of the result: its rows' codes, K and V, in the registers of a CTA, 16
// codes a thread and pass.
constexpr int kMoveThreads = 256;
constexpr int kMoveCluster = 8;
template <int D, int FMT, int PASSES>
struct MovedBlock {
  static constexpr int kLanes = D / 16, kRows = kMoveThreads / kLanes;
  uint4 code[2][PASSES];
  float scale[2][PASSES], mass[PASSES];
  float amax[2];
  int rows;
  bool moved;

  // reads the rows; every thread of the CTA gets the sides' largest values
  __device__ __forceinline__ void read(const EvictParams& p, int b, int h, int blk, int m,
                                       const int32_t* kept, uint32_t* red) {
    const Kv8& s = p.src;
    const int b0 = blk << p.dst.block_shift;
    rows = min(1 << p.dst.block_shift, m - b0);
    const int sub = threadIdx.x / kLanes, ch = (threadIdx.x % kLanes) * 16;
    bool other = false;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * kRows + sub;
      mass[i] = 0.0f;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        code[side][i] = make_uint4(0, 0, 0, 0);
        scale[side][i] = 0.0f;
      }
      if (r >= rows) continue;
      const int from = kept[b0 + r];
      other |= from != b0 + r;
      int in_page;
      const int page = kv8_page(s, b, from, in_page);
      if (page < 0) {
        set_status(p.status, CSA2_DEV_BAD_PAGE);
        continue;
      }
      const int64_t row = kv8_row(s, page, h, in_page), at = kv8_block(s, page, h, in_page);
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        code[side][i] = *reinterpret_cast<const uint4*>(s.codes[side] + row * D + ch);
        scale[side][i] = s.scales[side][at];
      }
      mass[i] = s.mass[row];
    }
    moved = __syncthreads_or(other);
    if (!moved) return;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      float big = 0.0f;
#pragma unroll
      for (int i = 0; i < PASSES; ++i)
        big = fmaxf(big, kv8_mag<FMT>(kv8_max16<FMT>(code[side][i])) * scale[side][i]);
      // magnitudes compare as their bits do
      amax[side] = __uint_as_float(group_max<kMoveThreads>(__float_as_uint(big), red, threadIdx.x));
    }
  }
  __device__ __forceinline__ void write(const EvictParams& p, int b, int h, int blk) {
    const Kv8& d = p.dst;
    int din;
    const int page = kv8_page(d, b, blk << d.block_shift, din);
    if (page < 0) {
      if (threadIdx.x == 0) set_status(p.status, CSA2_DEV_BAD_PAGE);
      return;
    }
    const int64_t drow = kv8_row(d, page, h, din), at = kv8_block(d, page, h, din);
    const int sub = threadIdx.x / kLanes, ch = (threadIdx.x % kLanes) * 16;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const float s1 = moved ? kv8_scale_of<FMT>(amax[side]) : 0.0f, inv = kv8_inverse(s1);
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = i * kRows + sub;
        if (r >= rows) continue;
        uint4 w = code[side][i];
        // A code that is not 0 is at least 2^-9 and the new scale at least its
        // value / 448, so f stays below 2^18.  A zero row does not bear on the new
        // scale and knows no such bound: held below f16's infinity, times which it
        // would not be 0.
        const float f = fminf(scale[side][i] * inv, 0x1p17f);
        if (moved && f != 1.0f) {
          // beyond f16's range (E4M3: rows of the smallest codes and zero rows) in
          // two steps, the first of which is exact
          const bool far = f > 32768.0f;
          if (far) w = recode16<FMT>(w, kv8_ratio(32768.0f));
          w = recode16<FMT>(w, kv8_ratio(far ? f * 0x1p-15f : f));
        }
        *reinterpret_cast<uint4*>(d.codes[side] + (drow + r) * D + ch) = w;
        if (side == 0 && ch == 0 && d.mass) d.mass[drow + r] = mass[i];
        if (r == 0 && ch == 0) d.scales[side][at] = moved ? s1 : scale[side][i];
      }
    }
  }
};

// Into another cache: one CTA per (block, head, sequence).  In place: a cluster
// per (head, sequence) walks the blocks upwards, one block a CTA and round; it
// reads a round's rows, meets at the cluster's barrier, and writes them.  A kept
// row never moves to a later place, so the sources of the rounds still to come
// lie behind the rows being written.  4096 rows kept of each of 4 sequences and 8
// heads, D 128, into another cache: 15 us, the rows' scattered halves of a
// kilobyte each.
template <int D, int FMT, int PASSES, bool PLACE>
__global__ void __launch_bounds__(kMoveThreads) kv8_evict_move_kernel(EvictParams p) {
  __shared__ uint32_t red[kMoveThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.y, b = blockIdx.z;
  const int n = p.old_len[b], m = min(n, p.keep);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.dst.seq_len[b] = m;
  const int32_t* kept = p.kept + ((int64_t)b * p.src.heads + h) * p.keep;
  const int blocks = (m + (1 << p.dst.block_shift) - 1) >> p.dst.block_shift;
  MovedBlock<D, FMT, PASSES> x;
  if (!PLACE) {
    if ((int)blockIdx.x >= blocks) return;
    x.read(p, b, h, blockIdx.x, m, kept, red);
    x.write(p, b, h, blockIdx.x);
    return;
  }
  if (n == m) return;                              // uniform over the cluster
  for (int first = 0; first < blocks; first += kMoveCluster) {
    const int blk = first + (int)blockIdx.x;       // the cluster is the grid's x
    const bool mine = blk < blocks;
    if (mine) x.read(p, b, h, blk, m, kept, red);
    cluster_sync();
    if (mine && x.moved) x.write(p, b, h, blk);
  }
}

template <typename... A>
cudaError_t launch_cluster(void (*kern)(A...), dim3 grid, int threads, int cluster, cudaStream_t s,
                           A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, int FMT, int PASSES>
cudaError_t move_as(const EvictParams& p, cudaStream_t s) {
  const int blocks = (p.keep + (1 << p.dst.block_shift) - 1) >> p.dst.block_shift;
  const dim3 grid(p.in_place ? kMoveCluster : blocks, p.src.heads, p.src.batch);
  return p.in_place ? launch_cluster(kv8_evict_move_kernel<D, FMT, PASSES, true>, grid, kMoveThreads,
                                     kMoveCluster, s, p)
                    : kv8_launch(kv8_evict_move_kernel<D, FMT, PASSES, false>, grid, kMoveThreads, 0,
                                 s, p);
}
template <int D, int FMT>
cudaError_t move_of(const EvictParams& p, cudaStream_t s) {
  constexpr int kMost = 128 * (D / 16) / kMoveThreads;   // passes of 128 rows
  switch (p.dst.block_shift) {
    case 7: return move_as<D, FMT, kMost>(p, s);
    case 6: return move_as<D, FMT, kMost / 2>(p, s);
    default: return move_as<D, FMT, (kMost > 3 ? kMost / 4 : 1)>(p, s);
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8& c, int D, const Kv8Rows& k, const Kv8Rows& v, int T,
                              const int32_t* new_len, const int32_t* start, uint32_t* status,
                              cudaStream_t s) {
  AppendParams p{c, {k, v}, T, new_len, start, status, 0};
  if (c.format == CSA2_KV8_E4M3)
    return D == 64 ? append_of<64, CSA2_KV8_E4M3>(p, s) : append_of<128, CSA2_KV8_E4M3>(p, s);
  return D == 64 ? append_of<64, CSA2_KV8_INT8>(p, s) : append_of<128, CSA2_KV8_INT8>(p, s);
}

cudaError_t launch_kv8_evict(const Kv8& src, const Kv8& dst, bool in_place, int D, int keep,
                             int sink, int recent, int32_t* kept, int32_t* old_len,
                             uint32_t* status, int num_sms, cudaStream_t s) {
  EvictParams p{src, dst, keep, sink, recent, kept, old_len, status, in_place ? 1 : 0};
  // CTAs per (head, sequence): as many as the SMs hold at once, up to eight and
  // one for each 2048 rows of the capacity
  int cluster = 8;
  while (cluster > 1 && ((int64_t)cluster * src.heads * src.batch > num_sms ||
                         src.max_len < 2048 * cluster))
    cluster /= 2;
  cudaError_t e = launch_cluster(kv8_evict_select_kernel, dim3(cluster, src.heads, src.batch),
                                 kSelThreads, cluster, s, p);
  if (e != cudaSuccess) return e;
  if (src.format == CSA2_KV8_E4M3)
    return D == 64 ? move_of<64, CSA2_KV8_E4M3>(p, s) : move_of<128, CSA2_KV8_E4M3>(p, s);
  return D == 64 ? move_of<64, CSA2_KV8_INT8>(p, s) : move_of<128, CSA2_KV8_INT8>(p, s);
}

}  // namespace csa2
