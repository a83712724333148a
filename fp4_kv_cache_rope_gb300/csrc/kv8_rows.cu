// The 8-bit K/V cache's append and eviction: rows into blocks of codes, and the
// rows that stay, moved into new blocks.  Both move bytes: their floor is the rows
// read once and written once.
#include "kv8_append.cuh"

namespace csa2 {
namespace {

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
  const AppendParams p{c, {k, v}, T, new_len, start, status, 0, nullptr, 0};
  return append_any<false>(p, D, s);
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
