// The weight that each cached row got from many query rows (a prompt's), on the
// tcgen05 tensor cores:
//
//   mass_j = decay mass_j + sum_r 2^(c q_r . k_j log2(e) - lse_r log2(e))
//
// The cached rows are M, so that a thread owns one of them and its sum needs no
// exchange: S^T [128 cached rows x kCols queries] = K Q^T, then one exponential
// and two additions per element.  A CTA turns its 128 rows of codes into an
// operand tile once and streams the queries that see them, 256 or 128 at a time;
// queries go in as they are (16-bit), K in their type: a code times its block's
// scale over the largest of the tile, a power of two, which is exact in bf16 and
// in f16 unless that is 2^-15 or less (then off by at most 2^-24 of the largest
// value).  2 D flop per pair against one exponential.  A prompt of 4096 tokens,
// 32 heads, D 128: 82 us; its products are 37 us at a library product's
// rate, its exponentials 29 us at 32 a cycle and SM.  The CTA with the most tiles
// has 64 for a mean of 56, and a tile takes 2400 cycles, in which its 64 KB of
// queries are copied 16 bytes at a time.
//
// x = fma(s, f, -a) with a fp32 constant per query.  f = c log2(e) is rounded,
// f = (1 - eps) true f: with a = (1 - eps) lse log2(e), rounded once, what is left
// is eps x, nothing for the weights that count.  (As two constants, -a and a
// factor of the sum for a's own rounding, 3e-7 of a weight at lse 14, the shared
// memory reads cost 7%.)
//
// The accumulation of S cuts off instead of rounding: over random sums a chain of
// k steps came out k 16 2^-31 of it too small (4 steps 4e-8, 8 steps 6.5e-8), which
// f makes up for; and with few queries D 128 goes in two chains that are added
// here.  Errors (norm): 55 tokens of 8 heads on 61176 rows 3.1e-6 as it is, 1.7e-6
// made up for, 1.1e-6 in two chains, 1.2e-6 by rounded fp32 sums; 1249 tokens of 4
// heads 1.0e-6, 0.31e-6, 0.20e-6, 0.23e-6.  Sums whose products share a sign lose
// two to four times as much, so that a part of it is left (logits of 35, bf16, two
// chains: 7.9e-7 as it is, 4.3e-7 made up for; f16, one chain: 4.6e-6, 2.6e-6).
//
// A cached row is one thread's in each of four warp groups: even and odd query
// tiles, left and right half of their columns.  Their four sums are added in a
// fixed order and written by a group that has the item's first query tile, so
// that items of a single tile alternate between two pairs of groups.
//
// Warps (768 threads): 0-15 exponentials; 16-19 copy queries (16 bytes at a
// time, asynchronously, into a ring); 20-22 turn K's codes into one of two
// operand tiles; 23 issues the MMAs.  With few query tiles to an item it is the
// loading that takes the time: hence a second K tile, warps of its own for K and
// an item's codes asked for one item ahead.  100 tokens of 4 heads on 8 caches of
// 16384 rows take 72 us (120 us before these three), 90 tokens of 2 on 21 of
// 120721 849 us (1312 us).
#include <type_traits>

#include "kv8_mma.cuh"

namespace csa2 {
namespace {

constexpr int kKeys = 128;
static_assert(kKeys == kKv8Step, "the items are the steps of the split");
constexpr double kCutOff = 1.0 / 2147483648.0;
constexpr int kExpWarps = 16;
constexpr int kQWarps = 4;
constexpr int kKWarps = 3;
constexpr int kThreads = 32 * (kExpWarps + kQWarps + kKWarps + 1);   // 80 registers each

template <int D, int ACCS>
struct MassSmem {
  static constexpr int kSlabs = D / 64;
  static constexpr int kCols = 256 / ACCS;            // queries of a tile
  static constexpr int kStages = 2 * ACCS, kConsts = 2 * kStages;
  static constexpr int kKSlab = kKeys * 128;          // [128 rows x 64 channels], swizzled
  static constexpr int kQSlab = kCols * 128;
  static constexpr int kK = 0;                        // 2 stages
  static constexpr int kQ = 2 * kSlabs * kKSlab;      // kStages
  static constexpr int kCode = kQ + kStages * kSlabs * kQSlab;   // the next item's codes, by chunk
  static constexpr int kConst = kCode + kKeys * kSlabs * 64;   // [kConsts][kCols] -a
  static constexpr int kSum = kConst + kConsts * kCols * 4;   // [2][3][128]
  static constexpr int kBars = kSum + 2 * 3 * kKeys * 4;
  static constexpr int kFlags = kBars + 192;          // abort, tmem, K's reference scale [4]
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
// The sequence of the last item looked up, and its items [before, end): the next
// one mostly lies in it too.
struct Seq {
  int b, n, ql;
  int64_t before, end;
};
template <int kCols>
__device__ __forceinline__ Item item_of(const MassParams& p, int lane, int64_t id, Seq& s) {
  const Kv8& c = p.a.c;
  if (id >= s.end) {
    s.b = kv8_find(c, lane, c.heads, id, s.before);
    s.n = kv8_len(c, s.b);
    s.end = s.before + (int64_t)kv8_steps(c, s.b) * c.heads;
    const int ql = p.a.q_len ? p.a.q_len[s.b] : p.a.T;
    s.ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
  }
  Item it;
  const int k = (int)(id - s.before);
  it.b = s.b;
  it.n = s.n;
  it.ql = s.ql;
  it.h = k % c.heads;
  it.key0 = k / c.heads * kKeys;
  it.rows = it.ql * p.a.G;
  const int tok0 = max(0, it.key0 - (it.n - it.ql));   // the first query that sees row key0
  it.first = tok0 * p.a.G / kCols;
  const int all = (it.rows + kCols - 1) / kCols;
  it.nt = it.key0 < it.n && tok0 < it.ql ? all - it.first : 0;
  return it;
}

// Sixteen codes times a power of two, in the queries' type.  bf16: a code as f16
// has at most eight significant bits and an exponent field of five that is not
// zero, so its bits moved down by three are a bf16 2^112 too small.
template <int FMT, typename V>
__device__ __forceinline__ void codes_to(uint4 w, float fs, uint32_t (&o)[8]) {
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h[2];
    kv8_to_f16<FMT>(ww[j], h[0], h[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (std::is_same<V, __nv_bfloat162>::value) {
        const uint32_t u = (h[e] >> 3 & 0x0FFF0FFFu) | (h[e] & 0x80008000u);
        const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                            __float2bfloat162_rn(fs * 5.19229686e33f));
        o[2 * j + e] = *reinterpret_cast<const uint32_t*>(&x);
      } else {
        const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h[e]), __float2half2_rn(fs));
        o[2 * j + e] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
  }
}

template <int D, int ACCS, int FMT>
__global__ void __launch_bounds__(kThreads, 1) kv8_mass_many_kernel(MassParams p) {
  using L = MassSmem<D, ACCS>;
  constexpr int kCols = L::kCols, kStages = L::kStages, kConsts = L::kConsts;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kMmaWarp = kExpWarps + kQWarps + kKWarps;
  const Kv8& c = p.a.c;
  griddep_wait();
  griddep_launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) set_status(p.a.status, CSA2_DEV_BAD_ALIGN);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* k_full = bars;        // [2] 3 warps, one phase per item
  uint64_t* k_empty = bars + 2;   // [2] commit of the item's last MMA
  uint64_t* q_full = bars + 4;    // [2 or 4] 4 warps
  uint64_t* q_empty = bars + 8;   // [2 or 4] commit
  uint64_t* s_full = bars + 12;   // [2] commit
  uint64_t* s_empty = bars + 14;  // [2] 8 warps
  uint64_t* x_full = bars + 16;   // [2] 12 warps: the other groups' sums of a round are there
  uint64_t* x_empty = bars + 18;  // [2] 4 warps: ... were read
  uint64_t* drain = bars + 20;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kFlags);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kFlags + 4);
  volatile float* refs = reinterpret_cast<volatile float*>(smem + L::kFlags + 8);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, kKWarps);
      mbar_init(k_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(s_empty + i, 8);
      mbar_init(x_full + i, 12);
      mbar_init(x_empty + i, 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(q_full + i, kQWarps);
      mbar_init(q_empty + i, 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, 512);
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
  Seq seq{0, 0, 0, 0, 0};
  if (warp < kExpWarps) {
    // ======================================================== exponential warps
    const int wg = warp >> 2, buf = wg >> 1, half = wg & 1, key = 32 * (warp & 3) + lane;
    const uint32_t tS =
        tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256 * buf + kCols / 2 * half;
    constexpr int kChunk = 32 / ACCS;   // columns read at a time
    float* sums = reinterpret_cast<float*>(smem + L::kSum);
    for (int64_t id; (id = item_id(round)) >= 0; ++round) {
      const Item it = item_of<kCols>(p, lane, id, seq);
      uint64_t acc[2] = {0, 0};
      // query rows below this one do not see the thread's cached row
      const int64_t see = (int64_t)(it.key0 + key - (it.n - it.ql)) * p.a.G;
      bool got = false;
      float f = 0.0f;
      // (the page's entry is asked for before the queries, and the weight before
      // the other groups' sums)
      const int other_wg = (wg - 2 * (int)(q & 1)) & 3;   // 0: this one writes
      const bool mine = other_wg == 0 && it.key0 + key < it.n;
      const int id_ = mine ? kv8_page_id(c, it.b, it.key0 + key) : 0;
      for (int i = 0; i < it.nt; ++i, ++q) {
        if ((q & 1) != (uint32_t)buf) continue;
        wait(s_full + buf, (q >> 1) & 1);
        tc_fence_after();
        if (!ok) break;
        if (!got) {
          got = true;
          // (K's tile of the item after next is not converted before this item's
          // last MMAs, and these warps are two query tiles behind at most: four slots)
          f = p.a.scale_log2 * refs[k & 3];
        }
        const float* cst = reinterpret_cast<const float*>(smem + L::kConst) + kCols * (q % kConsts) + kCols / 2 * half;
        const uint64_t f2 = pack2(f, f);
        const int64_t hid64 = see - (int64_t)(it.first + i) * kCols - kCols / 2 * half;
        const int hidden = hid64 < 0 ? 0 : (hid64 > kCols ? kCols : (int)hid64);
        auto add = [&](auto masked, int u) {
          uint32_t s[2][16];
          tmem_ld16(tS + kChunk * u, s[0]);
          tmem_ld16(tS + kChunk * u + (ACCS == 2 ? kCols : 16), s[1]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(s[0][j]), "+r"(s[1][j]));
          auto logits = [&](int j) {   // j and j + 1 of the chunk
            const uint32_t(&a)[16] = s[ACCS == 2 ? 0 : j >> 4];
            const uint64_t x = pack2(__uint_as_float(a[j & 15]), __uint_as_float(a[(j & 15) + 1]));
            if (ACCS == 1) return x;
            return add2(x, pack2(__uint_as_float(s[1][j & 15]), __uint_as_float(s[1][(j & 15) + 1])));
          };
#pragma unroll
          for (int j = 0; j < kChunk; j += 4) {
            const float4 h = *reinterpret_cast<const float4*>(cst + kChunk * u + j);
            const uint64_t hh[2] = {pack2(h.x, h.y), pack2(h.z, h.w)};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x, y;
              unpack2(fma2(logits(j + 2 * e), f2, hh[e]), x, y);
              x = kv8_exp2(x);
              y = kv8_exp2(y);
              if (decltype(masked)::value) {
                if (kChunk * u + j + 2 * e < hidden) x = 0.0f;
                if (kChunk * u + j + 2 * e + 1 < hidden) y = 0.0f;
              }
              acc[e] = add2(pack2(x, y), acc[e]);
            }
          }
        };
        // chunks of columns with a query in them
        const int chunks = (it.rows - (it.first + i) * kCols - kCols / 2 * half + kChunk - 1) / kChunk;
        if (__any_sync(0xffffffffu, hidden > 0)) {
#pragma unroll 1
          for (int u = 0; u < kCols / 2 / kChunk; ++u) add(std::true_type{}, u);
        } else {
#pragma unroll
          for (int u = 0; u < kCols / 2 / kChunk; ++u)
            if (u < chunks) add(std::false_type{}, u);
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
      if (other_wg > 0) {
        if (round >= 2) wait(x_empty + (round & 1), ((round >> 1) - 1) & 1);
        if (!ok) break;
        slot[(other_wg - 1) * kKeys] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(x_full + (round & 1));
        continue;
      }
      float* m = nullptr;
      float old = 0.0f;
      if (mine) {
        const int page = kv8_check(c, id_);
        if (page >= 0) {
          int in_page;
          kv8_in_page(c, it.key0 + key, in_page);
          m = c.mass + kv8_row(c, page, it.h, in_page);
          if (p.a.decay != 0.0f) old = *m;
        } else {
          set_status(p.a.status, CSA2_DEV_BAD_PAGE);
        }
      }
      wait(x_full + (round & 1), (round >> 1) & 1);
      if (!ok) break;
      const float other = (slot[0] + slot[kKeys]) + slot[2 * kKeys];
      __syncwarp();
      if (lane == 0) mbar_arrive(x_empty + (round & 1));
      if (m) {
        const float w = sum + other;
        *m = p.a.decay == 0.0f ? w : old * p.a.decay + w;
      }
    }
  } else if (warp < kExpWarps + kQWarps) {
    // ============================================================ query warps
    const int ct = tid - 32 * kExpWarps;
    const float eps = p.a.scale_low / p.a.scale_log2;
    for (int64_t id; (id = item_id(round)) >= 0; ++round) {
      const Item it = item_of<kCols>(p, lane, id, seq);
      if (it.nt == 0) continue;
      // A stage is free once its MMAs are done.  The constants' slots are twice as
      // many: the MMAs of tile q - kStages waited for the sums of the one two before.
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
      // A warp copies rows 4 w .. 4 w + 3 of every 16 of a tile, 8 lanes a row, and
      // its lanes make the constants of the same rows, cr + 128 v: so a row without
      // weight is cleared by the warp that copied it.
      const int cr = 16 * (lane >> 2) + 4 * (ct >> 5) + (lane & 3);
      Place pq = place(r0 + (ct >> 3), st_, sh_), pl = place(r0 + cr, p.a.H, 1);
      const int64_t q_by = 16 / G * st_ + 16 % G * sh_, q_wrap = st_ - G * sh_;
      const int64_t l_by = 128 / G * (int64_t)p.a.H + 128 % G, l_wrap = p.a.H - G;
      const char* qsrc = static_cast<const char*>(p.a.q.data) +
                         2 * (it.b * p.a.q.sb + (int64_t)it.h * G * sh_ + 8 * (ct & 7));
      const float* lsrc = p.a.lse + (int64_t)it.b * p.a.T * p.a.H + it.h * G;
      const int dst = (ct >> 3) * 128 + (((ct & 7) ^ ((ct >> 3) & 7)) << 4);
      for (int i = 0; i < it.nt; ++i, ++q) {
        const int st = q % kStages;
        if (q >= kStages) wait(q_empty + st, (q / kStages - 1) & 1);
        if (!ok) break;
        float y[kCols / 128];   // (asked for before the queries' copies)
        const int held = (it.rows - pl.r + 127) >> 7;   // (the v's below it are query rows)
#pragma unroll
        for (int v = 0; v < kCols / 128; ++v) {
          y[v] = pl.r < it.rows ? lsrc[pl.off] : -INFINITY;
          step(pl, 128, g128, l_by, l_wrap);
        }
        const uint32_t stage = smem_u32(smem + L::kQ + st * L::kSlabs * L::kQSlab) + dst;
        auto copy = [&](int v, const char* from, uint32_t size) {
#pragma unroll
          for (int s = 0; s < L::kSlabs; ++s)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             stage + s * L::kQSlab + v * 2048),
                         "l"(from + 128 * s), "r"(size)
                         : "memory");
        };
        if (g16 == 0) {   // 16 rows on are whole tokens: fewer instructions (a prompt: 86 -> 82 us)
          const char* from = qsrc + 2 * pq.off;
          const int left = it.rows - pq.r;
#pragma unroll 4
          for (int v = 0; v < kCols / 16; ++v, from += 2 * q_by)
            copy(v, 16 * v < left ? from : qsrc, 16 * v < left ? 16u : 0u);
          pq.r += kCols;
          pq.off += kCols / 16 * q_by;
        } else {
#pragma unroll 1
          for (int v = 0; v < kCols / 16; ++v) {
            const bool in = pq.r < it.rows;
            copy(v, qsrc + (in ? 2 * pq.off : 0), in ? 16u : 0u);
            step(pq, 16, g16, q_by, q_wrap);
          }
        }
        float* cst = reinterpret_cast<float*>(smem + L::kConst) + kCols * (q % kConsts);
#pragma unroll
        for (int v = 0; v < kCols / 128; ++v) {
          float a = INFINITY;                   // no weight (as for a lse of +inf)
          if (fabsf(y[v]) != INFINITY) {
            const float hi = y[v] * 1.44269502f;
            a = hi + (fmaf(y[v], 1.44269502f, -hi) + y[v] * 1.92596299e-8f - eps * hi);
          }
          cst[cr + 128 * v] = -a;
        }
        // rows without weight: a NaN or an infinity in them would count all the same
        // (the vote is taken while the copies are on their way)
        bool gone = false;
#pragma unroll
        for (int v = 0; v < kCols / 128; ++v) gone |= v < held && fabsf(y[v]) == INFINITY;
        const bool clear = __any_sync(0xffffffffu, gone);
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (clear) {
          __syncwarp();
#pragma unroll
          for (int v = 0; v < kCols / 128; ++v) {
            if (!(v < held && fabsf(y[v]) == INFINITY)) continue;
#pragma unroll 1
            for (int k = 0; k < 8 * L::kSlabs; ++k)
              *reinterpret_cast<uint4*>(smem + L::kQ + (st * L::kSlabs + (k >> 3)) * L::kQSlab +
                                        (cr + 128 * v) * 128 + 16 * (k & 7)) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + st);
      }
      if (!ok) break;
    }
  } else if (warp < kMmaWarp) {
    // ============================================================== K warps
    // 16-byte chunks i = ct + 96 v of the item.  An item's codes are asked for
    // while the one before is converted (each thread into the place that it has
    // just read), its page and scales before that.
    const int ct = tid - 32 * (kExpWarps + kQWarps);
    const bool bf16 = p.a.q.type == CSA2_BF16;
    constexpr int kChunks = kKeys * L::kSlabs * 4;
    constexpr int kIters = (kChunks + 32 * kKWarps - 1) / (32 * kKWarps), kBatch = 4;
    const uint32_t code = smem_u32(smem + L::kCode);
    Item it;
    int64_t grow = -1;   // of the 16 rows lane & 7, or -1
    float gs = 0.0f;
    // the next item with queries
    auto meta = [&]() -> bool {
      for (;; ++round) {
        const int64_t id = item_id(round);
        if (id < 0) return false;
        it = item_of<kCols>(p, lane, id, seq);
        if (it.nt > 0) break;
      }
      ++round;
      grow = -1;
      gs = 0.0f;
      const int pos = it.key0 + 16 * (lane & 7);
      if (pos < it.n) {
        int in_page;
        const int page = kv8_page(c, it.b, pos, in_page);
        if (page >= 0) {
          grow = kv8_row(c, page, it.h, in_page);
          gs = c.scales[0][kv8_block(c, page, it.h, in_page)];
        }
      }
      return true;
    };
    auto ask = [&](int i) {   // chunk i = (row * kSlabs + half) * 4 + chunk (whole warp)
      const int row = i / (4 * L::kSlabs);
      const int64_t g = __shfl_sync(0xffffffffu, grow, (row >> 4) & 7);
      const bool in = i < kChunks && g >= 0 && it.key0 + row < it.n;
      if (i < kChunks)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(code + 16 * i),
                     "l"(c.codes[0] + (in ? (g + (row & 15)) * D + 16 * (i % (4 * L::kSlabs)) : 0)),
                     "r"(in ? 16u : 0u)
                     : "memory");
    };
    bool more = meta();
    if (more) {
#pragma unroll
      for (int v = 0; v < kIters; ++v) ask(ct + 32 * kKWarps * v);
    }
    while (more) {
      float ref = gs;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
      const float rel = gs * kv8_inverse(ref);
      more = meta();
      if (k >= 2) wait(k_empty + (k & 1), ((k >> 1) - 1) & 1);
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok) break;
      if (ct == 0) refs[k & 3] = ref;
      auto put = [&](auto type) {
        using V = decltype(type);
#pragma unroll
        for (int v0 = 0; v0 < kIters; v0 += kBatch) {
          uint4 w[kBatch];
#pragma unroll
          for (int v = 0; v < kBatch; ++v) {
            const int i = ct + 32 * kKWarps * (v0 + v);
            w[v] = i < kChunks ? *reinterpret_cast<const uint4*>(smem + L::kCode + 16 * i)
                               : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int v = 0; v < kBatch; ++v) {
            const int i = ct + 32 * kKWarps * (v0 + v), row = i / (4 * L::kSlabs);
            const float fs = __shfl_sync(0xffffffffu, rel, (row >> 4) & 7);
            uint32_t o[8];
            codes_to<FMT, V>(w[v], fs, o);
            uint8_t* slab = smem + L::kK + ((k & 1) * L::kSlabs + i / 4 % L::kSlabs) * L::kKSlab;
            if (i < kChunks) {
              st_swizzled(slab, row, 2 * (i & 3), make_uint4(o[0], o[1], o[2], o[3]));
              st_swizzled(slab, row, 2 * (i & 3) + 1, make_uint4(o[4], o[5], o[6], o[7]));
            }
          }
          if (more) {
#pragma unroll
            for (int v = 0; v < kBatch; ++v) ask(ct + 32 * kKWarps * (v0 + v));
          }
        }
      };
      if (bf16)
        put(__nv_bfloat162());
      else
        put(__half2());
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full + (k & 1));
      ++k;
    }
  } else {
    // ================================================================== MMA warp
    const uint32_t fmt = p.a.q.type == CSA2_BF16 ? 1u : 0u;
    const uint32_t idesc = instr_desc(fmt, fmt, false, false, kKeys, kCols);
    const uint64_t kd = smem_desc(smem_u32(smem + L::kK), 16, 1024, 2);
    const uint64_t qd = smem_desc(smem_u32(smem + L::kQ), 16, 1024, 2);
    bool issued = false;
    for (int64_t id; (id = item_id(round)) >= 0; ++round) {
      const Item it = item_of<kCols>(p, lane, id, seq);
      if (it.nt == 0) continue;
      wait(k_full + (k & 1), (k >> 1) & 1);
      for (int i = 0; i < it.nt; ++i, ++q) {
        const int st = q & 1, stage = q % kStages;
        wait(q_full + stage, (q / kStages) & 1);
        if (q >= 2) wait(s_empty + st, ((q >> 1) - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int s = 0; s < L::kSlabs; ++s)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16(tmem + 256 * st + kCols * (kk & (ACCS - 1)),
                      kd + (((k & 1) * L::kSlabs + s) * L::kKSlab + kk * 32) / 16,
                      qd + ((stage * L::kSlabs + s) * L::kQSlab + kk * 32) / 16, idesc,
                      s > 0 || kk >= ACCS ? 1u : 0u);
          mma_commit(q_empty + stage);
          mma_commit(s_full + st);
          if (i + 1 == it.nt) mma_commit(k_empty + (k & 1));
        }
        issued = true;
      }
      if (!ok) break;
      ++k;
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
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int ACCS, int FMT>
cudaError_t mass_as(const Kv8Attn& a, int ctas, cudaStream_t s) {
  auto kern = kv8_mass_many_kernel<D, ACCS, FMT>;
  constexpr int bytes = MassSmem<D, ACCS>::kBytes;
  static std::atomic<uint64_t> seen;
  const cudaError_t e = kv8_prepare(kern, bytes, seen);
  if (e != cudaSuccess) return e;
  MassParams p{a};
  const double f = ((double)a.scale_log2 + (double)a.scale_low) * (1.0 + D / ACCS * kCutOff);
  p.a.scale_log2 = (float)f;
  p.a.scale_low = (float)(f - (double)p.a.scale_log2);
  return kv8_launch(kern, dim3(ctas), kThreads, bytes, s, p);
}
template <int FMT>
cudaError_t mass_of(const Kv8Attn& a, int ctas, cudaStream_t s) {
  if (a.D == 64) return mass_as<64, 1, FMT>(a, ctas, s);
  // Two accumulators up to 512 query rows, where the weight of a row can come from
  // a few queries and with it all their logits' error: 3.2e-6 of the weights in
  // one, 1.3e-6 in rounded fp32 sums (90 tokens of 2 heads on 120721 rows); the time
  // is not longer, 849 us against 938 us.  With more the errors average, 0.3e-6 for a
  // prompt of 4096 in one, and tiles of 256 queries are faster: 82 against 105 us.
  return a.T * a.G <= 512 ? mass_as<128, 2, FMT>(a, ctas, s) : mass_as<128, 1, FMT>(a, ctas, s);
}

}  // namespace

cudaError_t launch_kv8_mass_many(const Kv8Attn& a, int num_sms, cudaStream_t s) {
  return a.c.format == CSA2_KV8_E4M3 ? mass_of<CSA2_KV8_E4M3>(a, num_sms, s)
                                     : mass_of<CSA2_KV8_INT8>(a, num_sms, s);
}

cudaError_t set_wait_limit_kv8_mass(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace csa2
