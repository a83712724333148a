// The weight that each cached row got from many query rows (a prompt's), on the
// tcgen05 tensor cores:
//
//   mass_j = decay mass_j + sum_r 2^(c q_r . k_j log2(e) - lse_r log2(e))
//
// The cached rows are M, so that a thread owns one of them and its sum needs no
// exchange: S^T [128 cached rows x 256 queries] = K Q^T, then one exponential
// and two additions per element.  A CTA turns its 128 rows of codes into an
// operand tile once and streams the queries that see them, 256 rows at a time;
// queries go in as they are (16-bit), K in their type: a code times a power of
// two is exact in both.  2 D flop per pair against one exponential: the tensor
// cores and the issue slots of the eight exponential warps are about even.
//
// x = fma(s, f, -a) with a fp32 constant per query.  f = c log2(e) is rounded,
// f = (1 - eps) true f: with a = (1 - eps) lse log2(e), rounded once, what is left
// is eps x, nothing for the weights that count.  (As two constants, -a and a
// factor of the sum for a's own rounding, 3e-7 of a weight at lse 14, the shared
// memory reads cost 7%.)
//
// A cached row is one thread's in each of four warp groups: even and odd query
// tiles, left and right half of their columns.  Their four sums are added in a
// fixed order and written by the first group.
//
// Warps (672 threads): 0-15 exponentials; 16-19 load (K into its tile, queries
// by 16-byte asynchronous copies into a two-stage ring); 20 issues the MMAs.
#include <type_traits>

#include "kv8_mma.cuh"

namespace csa2 {
namespace {

constexpr int kKeys = 128;
static_assert(kKeys == kKv8Step, "the items are the steps of the split");
constexpr int kCols = 256;
constexpr int kThreads = 672;
constexpr int kExpWarps = 16;

template <int D>
struct MassSmem {
  static constexpr int kSlabs = D / 64;
  static constexpr int kKSlab = kKeys * 128;          // [128 rows x 64 channels], swizzled
  static constexpr int kQSlab = kCols * 128;
  static constexpr int kK = 0;
  static constexpr int kQ = kSlabs * kKSlab;          // 2 stages
  static constexpr int kConst = kQ + 2 * kSlabs * kQSlab;   // [4][256] -a
  static constexpr int kSum = kConst + 4 * kCols * 4;   // [2][3][128]
  static constexpr int kBars = kSum + 2 * 3 * kKeys * 4;
  static constexpr int kFlags = kBars + 128;          // abort, tmem, K's reference scale [4]
  // tensor memory holds one CTA, so a second is kept off the SM
  static constexpr int kBytes = kFlags + 64 < 120 * 1024 ? 120 * 1024 : kFlags + 64;
};

struct MassParams {
  Kv8Attn a;
};

// One 128-row tile of a (sequence, head) and the query tiles that see it.
struct Item {
  int b, h, key0, n, ql, rows, first, nt;   // rows = ql * G; query tiles first .. first + nt
};
__device__ __forceinline__ Item item_of(const MassParams& p, int lane, int64_t id) {
  const Kv8& c = p.a.c;
  Item it;
  int64_t before;
  it.b = kv8_find(c, lane, c.heads, id, before);
  const int k = (int)(id - before);
  it.h = k % c.heads;
  it.key0 = k / c.heads * kKeys;
  it.n = kv8_len(c, it.b);
  int ql = p.a.q_len ? p.a.q_len[it.b] : p.a.T;
  it.ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
  it.rows = it.ql * p.a.G;
  const int tok0 = max(0, it.key0 - (it.n - it.ql));   // the first query that sees row key0
  it.first = tok0 * p.a.G / kCols;
  const int all = (it.rows + kCols - 1) / kCols;
  it.nt = it.key0 < it.n && tok0 < it.ql ? all - it.first : 0;
  return it;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) kv8_mass_many_kernel(MassParams p) {
  using L = MassSmem<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Kv8& c = p.a.c;
  griddep_wait();
  griddep_launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) set_status(p.a.status, CSA2_DEV_BAD_ALIGN);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* k_full = bars;        // 4 warps, one phase per item
  uint64_t* k_empty = bars + 1;   // commit of the item's last MMA
  uint64_t* q_full = bars + 2;    // [2] 4 warps
  uint64_t* q_empty = bars + 4;   // [2] commit
  uint64_t* s_full = bars + 6;    // [2] commit
  uint64_t* s_empty = bars + 8;   // [2] 8 warps
  uint64_t* x_full = bars + 10;   // [2] 12 warps: the other groups' sums of a round are there
  uint64_t* x_empty = bars + 12;  // [2] 4 warps: ... were read
  uint64_t* drain = bars + 14;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kFlags);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kFlags + 4);
  volatile float* refs = reinterpret_cast<volatile float*>(smem + L::kFlags + 8);
  if (tid == 0) {
    mbar_init(k_full, 4);
    mbar_init(k_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 4);
      mbar_init(q_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(s_empty + i, 8);
      mbar_init(x_full + i, 12);
      mbar_init(x_empty + i, 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kExpWarps + 4) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;   // this thread's view: false once a wait gave up
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, abort_flag)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
  };
  const int64_t total = kv8_total(c, lane) * c.heads;

  // Items go out in rounds, forwards and backwards in turn: the first tiles of a
  // sequence are seen by the most queries, so long and short ones pair up.  -1: no
  // more (a round that a CTA misses is its last).
  auto item_id = [&](uint32_t round) -> int64_t {
    const int64_t id = (int64_t)round * gridDim.x +
                       (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    return id < total ? id : -1;
  };
  // q counts the CTA's query tiles over all items, k its items with queries
  uint32_t q = 0, k = 0, round = 0;
  if (warp < kExpWarps) {
    // ======================================================== exponential warps
    const int wg = warp >> 2, buf = wg >> 1, half = wg & 1, key = 32 * (warp & 3) + lane;
    const uint32_t tS =
        tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kCols * buf + kCols / 2 * half;
    float* sums = reinterpret_cast<float*>(smem + L::kSum);
    for (int64_t id; (id = item_id(round)) >= 0; ++round) {
      const Item it = item_of(p, lane, id);
      uint64_t acc[2] = {0, 0};
      // query rows below this one do not see the thread's cached row
      const int64_t see = (int64_t)(it.key0 + key - (it.n - it.ql)) * p.a.G;
      bool got = false;
      float f = 0.0f;
      for (int i = 0; i < it.nt; ++i, ++q) {
        if ((q & 1) != (uint32_t)buf) continue;
        wait(s_full + buf, (q >> 1) & 1);
        tc_fence_after();
        if (!ok) break;
        if (!got) {
          got = true;
          // (the tile after next is not written before this warp group's next
          // query tile is done with, so four slots are enough)
          f = p.a.scale_log2 * refs[k & 3];
        }
        const float* cst = reinterpret_cast<const float*>(smem + L::kConst) + kCols * (q & 3) + kCols / 2 * half;
        const uint64_t f2 = pack2(f, f);
        const int64_t hid64 = see - (int64_t)(it.first + i) * kCols - kCols / 2 * half;
        const int hidden = hid64 < 0 ? 0 : (hid64 > kCols ? kCols : (int)hid64);
        auto add = [&](auto masked, int u) {
          uint32_t s[32];
          tmem_ld32(tS + 32 * u, s);
          tmem_ld_wait();
          reg_fence32(s);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 h = *reinterpret_cast<const float4*>(cst + 32 * u + j);
            const uint64_t hh[2] = {pack2(h.x, h.y), pack2(h.z, h.w)};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t s2 = pack2(__uint_as_float(s[j + 2 * e]), __uint_as_float(s[j + 2 * e + 1]));
              float x, y;
              unpack2(fma2(s2, f2, hh[e]), x, y);
              x = kv8_exp2(x);
              y = kv8_exp2(y);
              if (decltype(masked)::value) {
                if (32 * u + j + 2 * e < hidden) x = 0.0f;
                if (32 * u + j + 2 * e + 1 < hidden) y = 0.0f;
              }
              acc[e] = add2(pack2(x, y), acc[e]);
            }
          }
        };
        if (__any_sync(0xffffffffu, hidden > 0)) {
#pragma unroll 1
          for (int u = 0; u < kCols / 64; ++u) add(std::true_type{}, u);
        } else {
#pragma unroll
          for (int u = 0; u < kCols / 64; ++u) add(std::false_type{}, u);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty + buf);
      }
      if (!ok) break;
      k += it.nt > 0;
      float a0, a1, a2, a3;
      unpack2(acc[0], a0, a1);
      unpack2(acc[1], a2, a3);
      const float sum = (a0 + a1) + (a2 + a3);
      // (waits with a limit, not a named barrier: a warp may have given up)
      float* slot = sums + (round & 1) * 3 * kKeys + key;
      if (wg > 0) {
        if (round >= 2) wait(x_empty + (round & 1), ((round >> 1) - 1) & 1);
        if (!ok) break;
        slot[(wg - 1) * kKeys] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(x_full + (round & 1));
        continue;
      }
      wait(x_full + (round & 1), (round >> 1) & 1);
      if (!ok) break;
      const float other = (slot[0] + slot[kKeys]) + slot[2 * kKeys];
      __syncwarp();
      if (lane == 0) mbar_arrive(x_empty + (round & 1));
      if (it.key0 + key < it.n) {
        int in_page;
        const int page = kv8_page(c, it.b, it.key0 + key, in_page);
        if (page >= 0) {
          float* m = c.mass + kv8_row(c, page, it.h, in_page);
          const float w = sum + other;
          *m = p.a.decay == 0.0f ? w : *m * p.a.decay + w;
        } else {
          set_status(p.a.status, CSA2_DEV_BAD_PAGE);
        }
      }
    }
  } else if (warp < kExpWarps + 4) {
    // ============================================================ loading warps
    const int ct = tid - 32 * kExpWarps;
    const bool bf16 = p.a.q.type == CSA2_BF16;
    const float eps = p.a.scale_low / p.a.scale_log2;
    for (int64_t id; (id = item_id(round)) >= 0; ++round) {
      const Item it = item_of(p, lane, id);
      if (it.nt == 0) continue;
      // ---- K: 16-byte chunk cc (of a 64-channel half) of rows r4 + 32 v
      if (k > 0) wait(k_empty, (k - 1) & 1);
      if (!ok) break;
      {
        const int cc = ct & 3, r4 = ct >> 2;
        int64_t grow = -1;
        float gs = 0.0f;
        const int pos = it.key0 + 16 * (lane & 7);
        if (pos < it.n) {
          int in_page;
          const int page = kv8_page(c, it.b, pos, in_page);
          if (page >= 0) {
            grow = kv8_row(c, page, it.h, in_page);
            gs = c.scales[0][kv8_block(c, page, it.h, in_page)];
          }
        }
        float ref = gs;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
        gs *= kv8_inverse(ref);
        if (ct == 0) refs[k & 3] = ref;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int row = r4 + 32 * v;
          const int64_t g = __shfl_sync(0xffffffffu, grow, row >> 4);
          const float fs = __shfl_sync(0xffffffffu, gs, row >> 4);
          const bool in = g >= 0 && it.key0 + row < it.n;
#pragma unroll
          for (int s = 0; s < L::kSlabs; ++s) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (in)
              w = *reinterpret_cast<const uint4*>(c.codes[0] + (g + (row & 15)) * D + 64 * s + 16 * cc);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float x[4];
              kv8_to_f32<FMT>(ww[j], x);
              o[2 * j] = pack16(x[0] * fs, x[1] * fs, bf16 ? CSA2_BF16 : CSA2_F16);
              o[2 * j + 1] = pack16(x[2] * fs, x[3] * fs, bf16 ? CSA2_BF16 : CSA2_F16);
            }
            uint8_t* slab = smem + L::kK + s * L::kKSlab;
            st_swizzled(slab, row, 2 * cc, make_uint4(o[0], o[1], o[2], o[3]));
            st_swizzled(slab, row, 2 * cc + 1, make_uint4(o[4], o[5], o[6], o[7]));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full);
        ++k;
      }
      // ---- queries.  A stage is free once its MMA is done; the constants' four
      // slots are: the MMA of tile q - 2 waited for the sums of tile q - 4.
      // Query row r is token r / G, head r % G of the group: each thread keeps
      // the place of its next row of queries (they go up by 16) and of its next
      // row of constants (by 128).
      const int G = p.a.G, r0 = it.first * kCols, g16 = 16 % G, g128 = 128 % G;
      struct Place {
        int r, g;
        int64_t off;
      };
      auto place = [&](int r, int64_t per_tok, int64_t per_head) {
        return Place{r, r % G, r / G * per_tok + r % G * per_head};
      };
      const int64_t st_ = p.a.q.st, sh_ = p.a.q.sh;
      auto step = [&](Place& x, int by, int by_head, int64_t by_off, int64_t wrap) {
        x.r += by;
        x.g += by_head;
        x.off += by_off;
        if (x.g >= G) {
          x.g -= G;
          x.off += wrap;
        }
      };
      Place pq = place(r0 + (ct >> 3), st_, sh_), pl = place(r0 + ct, p.a.H, 1);
      const int64_t q_by = 16 / G * st_ + 16 % G * sh_, q_wrap = st_ - G * sh_;
      const int64_t l_by = 128 / G * (int64_t)p.a.H + 128 % G, l_wrap = p.a.H - G;
      const char* qsrc = static_cast<const char*>(p.a.q.data) +
                         2 * (it.b * p.a.q.sb + (int64_t)it.h * G * sh_ + 8 * (ct & 7));
      const float* lsrc = p.a.lse + (int64_t)it.b * p.a.T * p.a.H + it.h * G;
      const int dst = (ct >> 3) * 128 + (((ct & 7) ^ ((ct >> 3) & 7)) << 4);
      for (int i = 0; i < it.nt; ++i, ++q) {
        const int st = q & 1;
        if (q >= 2) wait(q_empty + st, ((q >> 1) - 1) & 1);
        if (!ok) break;
        const uint32_t stage = smem_u32(smem + L::kQ + st * L::kSlabs * L::kQSlab) + dst;
#pragma unroll 4
        for (int v = 0; v < kCols / 16; ++v) {
          const bool in = pq.r < it.rows;
          const char* from = qsrc + (in ? 2 * pq.off : 0);
          const uint32_t size = in ? 16u : 0u;
#pragma unroll
          for (int s = 0; s < L::kSlabs; ++s)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             stage + s * L::kQSlab + v * 2048),
                         "l"(from + 128 * s), "r"(size)
                         : "memory");
          step(pq, 16, g16, q_by, q_wrap);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        float* cst = reinterpret_cast<float*>(smem + L::kConst) + kCols * (q & 3);
#pragma unroll
        for (int v = 0; v < kCols / 128; ++v) {
          float a = INFINITY;                   // no weight
          if (pl.r < it.rows) {
            const float y = lsrc[pl.off];
            if (y != -INFINITY) {
              const float hi = y * 1.44269502f;
              a = hi + (fmaf(y, 1.44269502f, -hi) + y * 1.92596299e-8f - eps * hi);
            }
          }
          cst[ct + 128 * v] = -a;
          step(pl, 128, g128, l_by, l_wrap);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + st);
      }
      if (!ok) break;
    }
  } else {
    // ================================================================== MMA warp
    const uint32_t fmt = p.a.q.type == CSA2_BF16 ? 1u : 0u;
    const uint32_t idesc = instr_desc(fmt, fmt, false, false, kKeys, kCols);
    const uint64_t kd = smem_desc(smem_u32(smem + L::kK), 16, 1024, 2);
    const uint64_t qd = smem_desc(smem_u32(smem + L::kQ), 16, 1024, 2);
    bool issued = false;
    for (int64_t id; (id = item_id(round)) >= 0; ++round) {
      const Item it = item_of(p, lane, id);
      if (it.nt == 0) continue;
      wait(k_full, k & 1);
      ++k;
      for (int i = 0; i < it.nt; ++i, ++q) {
        const int st = q & 1;
        wait(q_full + st, (q >> 1) & 1);
        if (q >= 2) wait(s_empty + st, ((q >> 1) - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int s = 0; s < L::kSlabs; ++s)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16(tmem + kCols * st, kd + (s * L::kKSlab + kk * 32) / 16,
                      qd + (st * L::kSlabs * L::kQSlab + s * L::kQSlab + kk * 32) / 16, idesc,
                      (s | kk) ? 1u : 0u);
          mma_commit(q_empty + st);
          mma_commit(s_full + st);
          if (i + 1 == it.nt) mma_commit(k_empty);
        }
        issued = true;
      }
      if (!ok) break;
    }
    if (issued && lane == 0) {   // let every issued MMA land before tensor memory is freed
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
  }
  __syncwarp();
  if (!ok) set_status(p.a.status, CSA2_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == kExpWarps + 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int FMT>
cudaError_t mass_as(const MassParams& p, int ctas, cudaStream_t s) {
  auto kern = kv8_mass_many_kernel<D, FMT>;
  static std::atomic<uint64_t> seen;
  cudaError_t e = kv8_prepare(kern, MassSmem<D>::kBytes, seen);
  if (e != cudaSuccess) return e;
  return kv8_launch(kern, dim3(ctas), kThreads, MassSmem<D>::kBytes, s, p);
}

}  // namespace

cudaError_t launch_kv8_mass_many(const Kv8Attn& a, int num_sms, cudaStream_t s) {
  const MassParams p{a};
  if (a.c.format == CSA2_KV8_E4M3)
    return a.D == 64 ? mass_as<64, CSA2_KV8_E4M3>(p, num_sms, s)
                     : mass_as<128, CSA2_KV8_E4M3>(p, num_sms, s);
  return a.D == 64 ? mass_as<64, CSA2_KV8_INT8>(p, num_sms, s)
                   : mass_as<128, CSA2_KV8_INT8>(p, num_sms, s);
}

cudaError_t set_wait_limit_kv8_mass(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace csa2
