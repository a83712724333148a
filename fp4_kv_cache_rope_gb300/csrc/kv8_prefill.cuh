// Attention over the 8-bit K/V cache for many query rows (prompts, chunks of
// prompts) on the tcgen05 tensor cores.
//
// A CTA takes 256 query rows of one (sequence, K/V head): token-major rows
// (token, head of the group), two M = 128 tiles.  It walks the cached rows in
// tiles of 128:
//
//   S = Q K^T      M 128 x N 128 x K D, f16 operands from shared memory;
//   P = 2^(S - m)  by the softmax warps, one thread per query row, written to
//                  tensor memory over S as f16;
//   O += P V       A = P from tensor memory, B = V (row-major as it lies).
//
// With both query tiles in flight the tensor cores work on one while the
// exponentials of the other are taken.  The arithmetic per cached byte is
// 256 rows' worth, so the tensor cores (4 D flop per query row and cached row)
// bound it; converting a tile's codes to f16 is paid once per 256 query rows.
// 4096 tokens of 64 heads at the end of 16384 rows, D 128: 1.68 ms, 1.15 PFLOP/s
// (61% of a library product's burst rate).  A tile of 128 rows takes 4600 cycles,
// of which the MMAs are 2100; the rest is the chain logits, maximum,
// exponentials, P, of which two query tiles in flight hide only a part.
//
// Exactness.  Queries are scaled per row by a power of two into f16's range;
// codes are converted to f16 times their block's scale over the largest scale
// in the CTA's range (both powers of two), so one factor per query row, and
// none per cached row, is left for the softmax.  A block whose scale is 2^12
// below the largest still keeps every bit; below that a value is off by at most
// 2^-25 of that largest scale, i.e. by 2^-31 of the range's largest value.
// The running maximum is raised only when a base-2 logit exceeds it by 8 (the rare
// rescaling of O stays off the common path), and P is taken times 2^7: at most
// 2^15 (2^16 is f16's infinity), with f16's full precision down to 2^-21.  l is summed in
// fp32 from the unrounded weights.
//
// Warps (640 threads): 0-3 and 4-7 softmax of query tile 0 and 1; 8-11 turn K's
// codes into f16 tiles and 12-15 V's, from registers loaded one tile ahead (no
// raw copy in shared memory, whose bandwidth the MMAs need); 16 issues the MMAs.
//
// A softmax thread reads its row's 128 logits from tensor memory twice, 16 at a
// time with the next ones on their way: once for the maximum, once for the
// exponentials.  That keeps the roles within their registers: a spilled register is read
// back from L2, because L1 is left little beside the tiles.  (Slopes reload 60 bytes, 124 at
// D 64; a mask alone with INT8 codes at D 64 44.)
//
// Changed scores (KIND).  A window or a prefix changes which tiles a CTA walks and what is
// hidden in them.  A slope is a multiply-add in both readings of S, exact in the
// distance.  A cap keeps the order of a row's logits, so the maximum is taken of the
// plain ones and capped once; the second reading takes four logits at a time through a
// quotient of polynomials in packed arithmetic (two operations in two cycles of the
// FMA pipe, but one issue).  Both together are taken once and kept in tensor memory.
// 4096 tokens of 64 heads at the end of 16384 rows, D 128: 2.68 ms with a cap, 2.58 ms with
// slopes, 4.50 ms with both, 1.79 ms with a prefix, against 1.75 ms for the same call with
// none.  The two softmax warps of an SM partition run chains of dependent instructions and
// leave half of its issue slots unused.
#pragma once

#include <type_traits>

#include "kv8_mma.cuh"
#include "kv8_scores.cuh"

namespace csa2 {
namespace {

constexpr int kTileKeys = 128;
constexpr int kNone = -0x7FFFFFFF - 1;   // no page id
constexpr int kTileRows = 256;
constexpr int kThreads = 640;
// Registers a thread at launch, and after the split among the warp groups.
constexpr int kRegs = 96, kRegsSoftmax = 104, kRegsConvert = 96, kRegsMma = 80;
static_assert(2 * kRegsSoftmax + 2 * kRegsConvert + kRegsMma <= 5 * kRegs, "register split");

template <int D>
struct PreSmem {
  static constexpr int kSlab = 128 * 128;            // [128 rows x 64 channels] f16, swizzled
  static constexpr int kSlabs = D / 64;
  static constexpr int kQ = 0;                       // 2 query tiles
  static constexpr int kK = kQ + 2 * kSlabs * kSlab; // 2 stages
  static constexpr int kV = kK + 2 * kSlabs * kSlab;
  static constexpr int kMisc = kV + 2 * kSlabs * kSlab;
  static constexpr int kBars = kMisc;                // 32 mbarriers
  static constexpr int kFlags = kMisc + 256;         // abort, tmem, tile masks [4], reduce [8]
  // tensor memory holds one CTA, so a second is kept off the SM
  static constexpr int kBytes = kMisc + 512 < 120 * 1024 ? 120 * 1024 : kMisc + 512;
};

// What changes the logits: nothing; nothing but which rows count; a cap; a slope;
// both.
enum Kind { kPlain, kMasked, kCapped, kSloped, kBoth };

struct PreParams {
  Kv8Attn a;
  int32_t rows, row_tiles, splits;
  Kv8Scores sc;                                      // what changes the scores (SCORED)
};

template <int D, int FMT, int KIND>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefill_kernel(PreParams p) {
  using L = PreSmem<D>;
  constexpr bool SCORED = KIND != kPlain;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Kv8& c = p.a.c;
  // (waits first: a later kernel of the stream takes this one's end for that of
  // the kernels before it, too)
  griddep_wait();
  griddep_launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) set_status(p.a.status, CSA2_DEV_BAD_ALIGN);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* start = bars;            // the queries and K of tile 0: 12 warps
  uint64_t* kv_full = bars + 1;      // [2: tile parity] V of tile i and K of i + 1: 8 warps
  uint64_t* s_full = bars + 5;       // [2 query tiles][2: tile parity] commit
  uint64_t* p_full = bars + 9;       // [2 query tiles] 4 warps
  uint64_t* o_done = bars + 13;      // commit after the last MMA
  uint64_t* drain = bars + 14;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kFlags);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kFlags + 4);
  volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + L::kFlags + 8);
  volatile float* red = reinterpret_cast<volatile float*>(smem + L::kFlags + 32);   // [K, V][4]
  volatile float* refs = red + 8;    // [K, V] largest scale in the CTA's range


  // ---- this CTA's share: heads fastest, then key splits, sequences, row tiles
  // (the last rows, which see the most keys, first)
  int id = blockIdx.x;
  const int h = id % c.heads;
  id /= c.heads;
  const int split = id % p.splits;
  id /= p.splits;
  const int b = id % c.batch;
  const int rt = p.row_tiles - 1 - id / c.batch;
  const int n = kv8_len(c, b);
  int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
  ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
  const int row0 = rt * kTileRows;
  const int rows = min(kTileRows, ql * p.a.G - row0);
  if (rows <= 0) return;                                    // uniform over the CTA
  const int last_tok = (row0 + rows - 1) / p.a.G;
  int keys = max(0, min(n, n - ql + last_tok + 1));
  int all_tiles = (keys + kTileKeys - 1) / kTileKeys;
  Kv8Span span{};                                           // SCORED: the tiles' rows
  int prefix = 0;
  if constexpr (SCORED) {
    if (p.sc.prefix) prefix = p.sc.prefix[b];
    keys = max(0, p.sc.sees(n - ql + last_tok, n, prefix));
    span = kv8_span_of(p.sc, p.sc.parent ? n : n - ql + row0 / p.a.G, keys, n, kTileKeys);
    all_tiles = span.steps;
  }
  const int t0 = (int)((int64_t)all_tiles * split / p.splits);
  const int nt = (int)((int64_t)all_tiles * (split + 1) / p.splits) - t0;
  const int mts = rows > 128 ? 2 : 1;                       // query tiles with rows

  if (tid == 0) {
    mbar_init(start, 12);
    for (int i = 0; i < 2; ++i) {
      mbar_init(kv_full + i, 8);
      mbar_init(s_full + i, 1);
      mbar_init(s_full + 2 + i, 1);
      mbar_init(p_full + i, 4);
    }
    mbar_init(o_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 16) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // first row of tile i of this CTA
  auto row_of = [&](int i) {
    return SCORED ? span.row(t0 + i, kTileKeys) : (t0 + i) * kTileKeys;
  };
  bool ok = true;   // this thread's view: false once a wait gave up
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, abort_flag)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
  };

  if (warp < 8) {
    // ============================================================ softmax warps
    regs_inc<kRegsSoftmax>();
    const int mt = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + 128 * mt, tO = tmem + lanes + 256 + D * mt;
    const int r = 128 * mt + 32 * (warp & 3) + lane;       // this thread's query row
    const int gr = row0 + r, tok = gr / p.a.G, hd = h * p.a.G + gr % p.a.G;
    const bool real = r < rows;
    // (a row without a query is never written: it may see everything)
    int lim = real ? min(n, n - ql + tok + 1) : 0x7FFFFFFF;
    int low = -kNoQuery;                                   // SCORED: from here on, or below the sink
    float at = 0.0f, slope = 0.0f;                         // the query's position; base 2
    if (SCORED && real) {
      const int pos = kv8_query_at(p.a, p.sc, b, n, ql, tok);
      lim = p.sc.sees(pos, n, prefix);
      low = p.sc.from(pos);
      at = (float)pos;
      if (KIND == kSloped || KIND == kBoth) slope = p.sc.slopes[hd] * kLog2e;
    }
    float mul = 0.0f;
    constexpr int kPer = D / 8;                            // 16-byte chunks of a row
    constexpr int kAt = 32 / kPer;                         // rows of a warp's access
    const int chunk = lane % kPer;
    if (nt > 0) {
      // the warp's 32 rows as f16 in the swizzled tile, kAt rows an access
      const int64_t off = b * p.a.q.sb + tok * p.a.q.st + hd * p.a.q.sh;
      uint8_t* tile = smem + L::kQ + mt * L::kSlabs * L::kSlab + (chunk >> 3) * L::kSlab;
      float up = 1.0f;
#pragma unroll 8
      for (int i = 0; i < 32 / kAt; ++i) {
        const int row = i * kAt + lane / kPer;             // of the warp's 32
        const int64_t from = __shfl_sync(0xffffffffu, off, row);
        const bool in = __shfl_sync(0xffffffffu, (int)real, row) != 0;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (in)
          w = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.a.q.data) + 2 * from +
                                              16 * chunk);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        float x[8], amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (p.a.q.type == CSA2_BF16) {
            bf16x2_to_f32(ww[j], x[2 * j], x[2 * j + 1]);
          } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[j]));
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
          }
          amax = fmaxf(amax, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
        }
#pragma unroll
        for (int o = kPer / 2; o > 0; o >>= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e = (int)(__float_as_uint(amax) >> 23);
        const int shift = e == 0 || e == 255 ? 0 : 134 - e;
        const float f = __uint_as_float((uint32_t)(127 + (shift > 127 ? 127 : shift)) << 23);
        const float mine = __shfl_sync(0xffffffffu, f, lane % kAt * kPer);
        if (lane / kAt == i) up = mine;
        st_swizzled(tile, 32 * (warp & 3) + row, chunk & 7,
                    make_uint4(pack16(x[0] * f, x[1] * f, CSA2_F16), pack16(x[2] * f, x[3] * f, CSA2_F16),
                               pack16(x[4] * f, x[5] * f, CSA2_F16), pack16(x[6] * f, x[7] * f, CSA2_F16)));
      }
      mul = (SCORED ? p.sc.factor : p.a.scale_log2) / up;   // times K's largest scale, below
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(start);
    }

    float m = -INFINITY;
    uint64_t l2[2] = {0, 0};                   // the sum, as four partial ones
    for (int i = 0; mt < mts && i < nt; ++i) {
      wait(s_full + 2 * mt + (i & 1), (i >> 1) & 1);
      tc_fence_after();
      if (!ok) break;
      if (i == 0) {
        // (kept above zero: hidden columns are -inf times it)
        const float kref = refs[0];
        mul = fmaxf(mul * (kref > 0.0f ? kref : 1.0f), 1.2e-38f);
      }
      // written before the tile's K was handed over, and not written again
      // before QK of tile i + 1, which waits for this tile's P
      const uint32_t groups = masks[i & 3];
      const int key0 = row_of(i);
      bool front = false;                                  // some row's window hides some
      if (SCORED && p.sc.window && key0 + kTileKeys > p.sc.sink)
        front = __any_sync(0xffffffffu, low > key0);
      const bool masked = groups != 0xFFu || front || __any_sync(0xffffffffu, lim < key0 + kTileKeys);
      const int seen = masked ? (int)__reduce_min_sync(0xffffffffu, max(lim - key0, 0)) : 0;
      // The columns 16 u .. that the row does not see, a bit each: kCapped hides them as 0,
      // which neither its size nor a score beside them tells, and then as -inf.  (By
      // comparisons twice, as below, a chunk of 4096 tokens took 2727 us, 2685 this way.)
      auto hidden = [&](int u) -> uint32_t {
        if (!((groups >> u) & 1u)) return 0xFFFFu;
        if (seen >= 16 * u + 16 && !front) return 0u;      // every row sees them
        const int x = key0 + 16 * u;
        uint32_t bits = 0xFFFFu << min(max(lim - x, 0), 16);
        if (front)
          bits |= ((1u << min(max(low - x, 0), 16)) - 1u) & (0xFFFFu << min(max(p.sc.sink - x, 0), 16));
        return bits;
      };
      auto put = [&](uint32_t (&s)[16], uint32_t bits, uint32_t with) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (bits >> j & 1u) s[j] = with;
      };
      constexpr uint32_t kMinusInf = 0xFF800000u;
      auto hide = [&](uint32_t (&s)[16], int u) {
        const bool gone = !((groups >> u) & 1u);
        if (!gone && seen >= 16 * u + 16 && !front) return;   // every row sees them
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (gone || key0 + 16 * u + j >= lim) s[j] = kMinusInf;
        if constexpr (SCORED) {
          if (!front) return;
          const int to = low - (key0 + 16 * u), from = p.sc.sink - (key0 + 16 * u);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < to && j >= from) s[j] = kMinusInf;
        }
      };
      // kSloped: logits in base 2, plus `add`; a row's bias is linear in the column
      // but where a prefix lets rows behind the query count
      bool mirrored = false;
      if (KIND == kSloped && p.sc.prefix)
        mirrored = __any_sync(0xffffffffu, at < (float)(key0 + kTileKeys - 1));
      auto sloped = [&](uint32_t (&s)[16], int u, float add, auto both) {
        const uint64_t f = pack2(mul, mul);
        const float d0 = (float)(key0 + 16 * u) - at;
        const uint64_t by = pack2(slope, slope), more = pack2(add, add);
        auto row = [&](uint64_t d, int j) {
          float x, y;
          unpack2(fma2(pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), f, fma2(d, by, more)), x, y);
          s[j] = __float_as_uint(x);
          s[j + 1] = __float_as_uint(y);
        };
        if constexpr (decltype(both)::value) {
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            row(pack2(-fabsf(d0 + (float)j), -fabsf(d0 + (float)(j + 1))), j);
        } else {
          uint64_t d = pack2(d0, d0 + 1.0f);               // exact, like every step
          const uint64_t two = pack2(2.0f, 2.0f);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            row(d, j);
            d = add2(d, two);
          }
        }
      };
      using Yes = std::integral_constant<bool, true>;
      using No = std::integral_constant<bool, false>;
      // kBoth: capped logits in base 2
      auto capped = [&](uint32_t (&s)[16]) {
        const uint64_t f = pack2(mul, mul);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float x, y;
          unpack2(mul2(pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), f), x, y);
          s[j] = __float_as_uint(kv8_cap(x, p.sc.cap2));
          s[j + 1] = __float_as_uint(kv8_cap(y, p.sc.cap2));
        }
      };
      // f(columns 16 u .., u) for u = 0 .. 7, the next ones on their way meanwhile
      auto each = [&](auto f) {
        uint32_t sa[16], sb[16];
        tmem_ld16(tS, sa);
        tmem_ld_wait();
        reg_fence(sa);
        // (what changes the scores takes so many instructions that eight copies of
        // them would be fetched anew each time: two of them for prompts of 64 channels
        // with slopes 46 us, four times two 53 us)
#pragma unroll KIND == kPlain || KIND == kMasked ? 4 : KIND == kBoth ? 1 : 2
        for (int u = 0; u < 8; u += 2) {
          tmem_ld16(tS + 16 * (u + 1), sb);
          f(sa, u);
          tmem_ld_wait();
          reg_fence(sb);
          if (u + 2 < 8) tmem_ld16(tS + 16 * (u + 2), sa);
          f(sb, u + 1);
          tmem_ld_wait();
          reg_fence(sa);
        }
      };
      // change, hide where some row does not see all, use: a loop of its own each way, for
      // a branch in every step costs more than the code
      auto pass = [&](auto change, auto use) {
        if (masked)
          each([&](uint32_t (&s)[16], int u) {
            if constexpr (KIND == kCapped) {
              // (scores that share a reciprocal with hidden ones)
              const uint32_t bits = hidden(u);
              put(s, bits, 0u);
              change(s, u);
              put(s, bits, kMinusInf);
            } else {
              change(s, u);
              hide(s, u);
            }
            use(s, u);
          });
        else
          each([&](uint32_t (&s)[16], int u) {
            change(s, u);
            use(s, u);
          });
      };
      float tops[2] = {-INFINITY, -INFINITY};
      auto largest = [&](uint32_t (&s)[16], int) {
#pragma unroll
        for (int j = 0; j < 16; j += 2)
          tops[(j >> 1) & 1] = KIND == kPlain
                                   ? fmaxf(tops[(j >> 1) & 1],
                                           fmaxf(__uint_as_float(s[j]), __uint_as_float(s[j + 1])))
                                   : max3(tops[(j >> 1) & 1], __uint_as_float(s[j]),
                                          __uint_as_float(s[j + 1]));
      };
      float size = 0.0f;                                   // kCapped: the largest |logit| seen
      if constexpr (KIND == kBoth) {
        // (taken once, and kept in tensor memory)
        pass(
            [&](uint32_t (&s)[16], int u) {
              capped(s);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                s[j] = __float_as_uint(fmaf(-slope, fabsf(at - (float)(key0 + 16 * u + j)), __uint_as_float(s[j])));
            },
            [&](uint32_t (&s)[16], int u) {
              largest(s, u);
              tmem_st16(tS + 16 * u, s);
            });
        tmem_st_wait();
      } else if constexpr (KIND == kSloped) {
        if (mirrored)
          pass([&](uint32_t (&s)[16], int u) { sloped(s, u, 0.0f, Yes{}); }, largest);
        else
          pass([&](uint32_t (&s)[16], int u) { sloped(s, u, 0.0f, No{}); }, largest);
      } else {
        if constexpr (KIND == kCapped) {
          auto measure = [&](const uint32_t (&s)[16]) {
#pragma unroll
            for (int j = 0; j < 16; j += 2)
              size = max3_abs(size, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
          };
          if (masked)
            each([&](uint32_t (&s)[16], int u) {
              const uint32_t bits = hidden(u);
              put(s, bits, 0u);
              measure(s);
              put(s, bits, kMinusInf);
              largest(s, u);
            });
          else
            each([&](uint32_t (&s)[16], int u) {
              measure(s);
              largest(s, u);
            });
        } else if (masked) {
          each([&](uint32_t (&s)[16], int u) {
            hide(s, u);
            largest(s, u);
          });
        } else {
          each(largest);
        }
      }
      // what the logits in tensor memory lack to base 2
      const float by = KIND == kSloped || KIND == kBoth ? 1.0f : mul;
      float top = fmaxf(tops[0], tops[1]) * by;
      if constexpr (KIND == kCapped) {
        // (the cap keeps their order; a row that sees nothing starts from the least score
        // that there is)
        top = kv8_cap(top, p.sc.cap2);
      }
      // (a row without a visible key so far waits for one; rows share nothing but, by
      // warp, which form of the arithmetic below takes their weights)
      // A capped score and its row's largest are each off by up to 4e-7 of the cap: one power
      // of two between them for a cap of 2^20.  So with large caps less of P's range is left
      // to the maximum's lag.
      const bool raise = top > m + (KIND == kCapped && p.sc.cap2 > 65536.0f ? 4.0f : 8.0f);
      if (__any_sync(0xffffffffu, raise)) {
        const float up = raise ? top : m;
        const float alpha = m == -INFINITY ? 0.0f : kv8_exp2(m - up);
        const uint64_t a2 = pack2(alpha, alpha);
        l2[0] = mul2(l2[0], a2);
        l2[1] = mul2(l2[1], a2);
        m = up;
        if (i > 0) {
          // (P V of the tile before was issued ahead of this tile's Q K^T, so O
          // is complete with S)
#pragma unroll 1
          for (int u = 0; u < D / 16; ++u) {
            uint32_t o[16];
            tmem_ld16(tO + 16 * u, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st16(tO + 16 * u, o);
          }
          tmem_st_wait();
        }
      }
      // One fused multiply-add gives the exponent: m's own rounding is then the
      // same for the whole row and cancels in P / l.  Where m is so large that
      // it would carry P out of range (ulp(2^16) = 2^-7), the logits are rounded
      // like m, which makes the largest difference 0 again.
      // kSloped rounds the bias with what is added to it, so the same goes for biases
      // beyond 2^20 (ulp 2^-3), which only logits as large make up for.
      const float mm = m == -INFINITY ? 0.0f : m;
      const float less = 7.0f - mm;
      const uint64_t f2 = pack2(by, by), u2 = pack2(less, less);
      auto weights = [&](uint32_t (&s)[16], int u) {        // exponents -> P
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = kv8_exp2(__uint_as_float(s[2 * j])), y = kv8_exp2(__uint_as_float(s[2 * j + 1]));
          l2[j & 1] = add2(l2[j & 1], pack2(x, y));
          w[j] = pack16(x, y, CSA2_F16);
        }
        tmem_st8(tS + 8 * u, w);
      };
      auto exponents = [&](uint32_t (&s)[16]) {
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float x, y;
          unpack2(fma2(pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), f2, u2), x, y);
          s[j] = __float_as_uint(x);
          s[j + 1] = __float_as_uint(y);
        }
      };
      bool large = fabsf(mm) > 65536.0f;
      if (KIND == kSloped)
        large |= fabsf(slope) * fmaxf(fabsf((float)key0 - at), fabsf((float)(key0 + kTileKeys) - at)) > 0x1p20f;
      if (KIND != kCapped && __any_sync(0xffffffffu, large)) {
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
          uint32_t s[16];
          tmem_ld16(tS + 16 * u, s);
          tmem_ld_wait();
          reg_fence(s);
          if constexpr (KIND == kSloped) sloped(s, u, 0.0f, Yes{});
          hide(s, u);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            s[j] = __float_as_uint((__fmul_rn(__uint_as_float(s[j]), by) - mm) + 7.0f);
          weights(s, u);
        }
      } else if constexpr (KIND == kCapped) {
        // By warp, so another row's scores may change a row's last bits; keys that none of
        // the warp's rows sees do not.  (Both quotients where a warp's rows differ, each row by
        // its own scores: 4096 tokens of 64 heads at the end of 16384 rows, D 128, scores around
        // twice the cap 4844 -> 6374 us, of the cap 3729 -> 9570 us.)
        const NearCap near(mul, p.sc.cap2);
        auto near4 = [&](uint32_t (&s)[16], int j, float (&x)[4]) {
          uint64_t a = pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1]));
          uint64_t c = pack2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
          near(a, c, u2);
          unpack2(a, x[0], x[1]);
          unpack2(c, x[2], x[3]);
        };
        auto far4 = [&](uint32_t (&s)[16], int j, float (&x)[4]) {
          const uint64_t f = pack2(mul, mul);
          unpack2(mul2(pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), f), x[0], x[1]);
          unpack2(mul2(pack2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), f), x[2], x[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = kv8_cap(x[k], p.sc.cap2, less);
        };
        auto by4 = [&](auto cap4) {
          pass(
              [&](uint32_t (&s)[16], int) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                  float x[4];
                  cap4(s, j, x);
#pragma unroll
                  for (int k = 0; k < 4; ++k) s[j + k] = __float_as_uint(x[k]);
                }
              },
              weights);
        };
        if (__all_sync(0xffffffffu, size * mul <= kTanhNear && mul <= kNearMul))
          by4(near4);
        else
          by4(far4);
      } else if constexpr (KIND == kSloped) {
        if (mirrored)
          pass([&](uint32_t (&s)[16], int u) { sloped(s, u, less, Yes{}); }, weights);
        else
          pass([&](uint32_t (&s)[16], int u) { sloped(s, u, less, No{}); }, weights);
      } else if (masked) {
        each([&](uint32_t (&s)[16], int u) {
          hide(s, u);
          exponents(s);
          weights(s, u);
        });
      } else {
        each([&](uint32_t (&s)[16], int u) {
          exponents(s);
          weights(s, u);
        });
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + mt);
    }
    float l = 0.0f;
    {
      float a, b2, c2, d;
      unpack2(l2[0], a, b2);
      unpack2(l2[1], c2, d);
      l = (a + b2) + (c2 + d);
    }
    // ---- the row's result
    if (nt > 0 && mt < mts) wait(o_done, 0);
    tc_fence_after();
    const bool empty = l == 0.0f;
    const float base2 = empty ? -INFINITY : m + log2f(l) - 7.0f;
    if (SCORED && p.splits == 1 && p.sc.rows_out) {
      // the drafted rows are still to come
      float* to = p.sc.rows_out + (((int64_t)b * p.a.T + (real ? tok : 0)) * p.a.H + hd) * kv8_row_floats(D);
      const float f = empty ? 0.0f : refs[1];
#pragma unroll
      for (int u = 0; u < D / 16; ++u) {
        uint32_t s[16];
        if (nt > 0 && mt < mts && ok) {
          tmem_ld16(tO + 16 * u, s);
          tmem_ld_wait();
          reg_fence(s);
        }
        if (!real || !ok) continue;
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(to + 16 * u + j) =
              empty ? make_float4(0, 0, 0, 0)
                    : make_float4(__uint_as_float(s[j]) * f, __uint_as_float(s[j + 1]) * f,
                                  __uint_as_float(s[j + 2]) * f, __uint_as_float(s[j + 3]) * f);
      }
      if (real) {
        to[D] = m - 7.0f;
        to[D + 1] = ok ? l : 0.0f;
      }
    } else if (p.splits == 1) {
      // through shared memory (the query tile, done with), so that a row's
      // stores go out together: 16-byte chunks, swizzled by the row
      const float f = empty ? 0.0f : refs[1] / l;
      uint8_t* stage = smem + L::kQ + warp * 32 * 2 * D;
#pragma unroll
      for (int u = 0; u < D / 16; ++u) {
        uint32_t s[16];
        if (nt > 0 && mt < mts && ok) {
          tmem_ld16(tO + 16 * u, s);
          tmem_ld_wait();
          reg_fence(s);
        }
#pragma unroll
        for (int j = 0; j < 16; j += 8) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = empty ? 0u
                         : pack16(__uint_as_float(s[j + 2 * q]) * f,
                                  __uint_as_float(s[j + 2 * q + 1]) * f, p.a.out.type);
          const int at = (2 * u + (j >> 3)) ^ (lane & 7);
          *reinterpret_cast<uint4*>(stage + lane * 2 * D + 16 * at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      const int64_t off = b * p.a.out.sb + tok * p.a.out.st + hd * p.a.out.sh;
#pragma unroll 4
      for (int i = 0; i < 32 / kAt; ++i) {
        const int row = i * kAt + lane / kPer;
        const int64_t to = __shfl_sync(0xffffffffu, off, row);
        const bool in = __shfl_sync(0xffffffffu, (int)(real && ok), row) != 0;
        if (in)
          *reinterpret_cast<uint4*>(static_cast<char*>(const_cast<void*>(p.a.out.data)) + 2 * to +
                                    16 * chunk) =
              *reinterpret_cast<const uint4*>(stage + row * 2 * D + 16 * (chunk ^ (row & 7)));
      }
      if (real && ok && p.a.lse)
        p.a.lse[((int64_t)b * p.a.T + tok) * p.a.H + hd] =
            empty ? -INFINITY : base2 * 0.6931471805599453f;
    } else {
      float* part = p.a.part + (int64_t)blockIdx.x * kTileRows * (D + 2);
      const float f = empty ? 0.0f : refs[1];
#pragma unroll
      for (int u = 0; u < D / 32; ++u) {
        uint32_t s[32];
        if (nt > 0 && mt < mts && ok) {
          tmem_ld32(tO + 32 * u, s);
          tmem_ld_wait();
          reg_fence32(s);
        }
        if (!real || !ok) continue;
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(part + r * D + 32 * u + j) =
              empty ? make_float4(0, 0, 0, 0)
                    : make_float4(__uint_as_float(s[j]) * f, __uint_as_float(s[j + 1]) * f,
                                  __uint_as_float(s[j + 2]) * f, __uint_as_float(s[j + 3]) * f);
      }
      if (real) {
        part[kTileRows * D + r] = m;
        part[kTileRows * (D + 1) + r] = ok ? l : 0.0f;
      }
    }
  } else if (warp < 16) {
    // ========================================================== converter warps
    // Thread: 16-byte chunk cc (of a 64-channel half) of rows r4 + 32 v.  Eight
    // neighbouring lanes then store to two rows' chunks of all eight positions.
    regs_dec<kRegsConvert>();
    const int side = warp >= 12, ct = tid & 127, cc = ct & 3, r4 = ct >> 2;
    constexpr int kPer = L::kSlabs * 4;
    uint8_t* tiles = smem + (side ? L::kV : L::kK);
    const uint8_t* codes = c.codes[side] + 16 * cc;
    const float* scales = c.scales[side];
    // ---- the side's largest scale in the range (a power of two; 0 when all are)
    float inv;
    {
      float mx = 0.0f;
      const int blk = 1 << c.block_shift, end = min(keys, (t0 + nt) * kTileKeys);
      if constexpr (SCORED) {
        const int shift = 7 - c.block_shift;   // blocks of a tile
#pragma unroll 4
        for (int i = ct; i < nt << shift; i += 128) {
          const int pos = row_of(i >> shift) + ((i & ((1 << shift) - 1)) << c.block_shift);
          int in_page;
          const int page = pos < keys ? kv8_page(c, b, pos, in_page) : -1;
          if (page >= 0) mx = fmaxf(mx, scales[kv8_block(c, page, h, in_page)]);
        }
      } else {
#pragma unroll 4
        for (int pos = t0 * kTileKeys / blk * blk + ct * blk; pos < end; pos += 128 * blk) {
          int in_page;
          const int page = kv8_page(c, b, pos, in_page);
          if (page >= 0) mx = fmaxf(mx, scales[kv8_block(c, page, h, in_page)]);
        }
      }
      // scales are not negative: their bits compare alike
      mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
      if (lane == 0) red[4 * side + (warp & 3)] = mx;
      bar_sync(1 + side, 128);                 // (nothing before it can give up)
      mx = fmaxf(fmaxf(red[4 * side], red[4 * side + 1]), fmaxf(red[4 * side + 2], red[4 * side + 3]));
      if (ct == 0) refs[side] = mx;
      inv = kv8_inverse(mx);
    }
    // Lanes 0..7 look after the tile's eight 16-row groups.  A warp stops at the
    // first use of a value that is still on its way, so each lookup is a tile
    // apart from the next: page ids three tiles ahead, rows and scales two, codes
    // one.
    int in_page = 0;
    auto fetch = [&](int i) -> int {         // page id; kNone: no row of this group counts
      if (SCORED && i >= nt) return kNone;
      const int pos = row_of(i) + 16 * (lane & 7);
      if (i >= nt || pos >= keys) return kNone;
      return kv8_page_id(c, b, pos);
    };
    int64_t grow = -1;
    float gs = 0.0f;
    auto place = [&](int i, int id) {
      grow = -1;
      gs = 0.0f;
      if (id == kNone) return;
      const int page = kv8_check(c, id);
      if (page >= 0) {
        kv8_in_page(c, row_of(i) + 16 * (lane & 7), in_page);
        grow = kv8_row(c, page, h, in_page);
        gs = scales[kv8_block(c, page, h, in_page)];
      } else if (lane < 8) {
        set_status(p.a.status, CSA2_DEV_BAD_PAGE);
      }
    };
    uint4 raw[kPer];
    float fac[4];
    auto load = [&](int i) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = r4 + 32 * v;
        const int64_t g = __shfl_sync(0xffffffffu, grow, row >> 4);
        fac[v] = __shfl_sync(0xffffffffu, gs, row >> 4) * inv;
        // rows the CTA does not see stay 0: their scales are not in the range
        const bool in = g >= 0 && row_of(i) + row < keys;
        const uint8_t* from = codes + (g + (row & 15)) * D;
#pragma unroll
        for (int s = 0; s < L::kSlabs; ++s) {
          raw[s * 4 + v] = make_uint4(0, 0, 0, 0);
          if (in) raw[s * 4 + v] = load_once(from + 64 * s);
        }
      }
    };
    auto convert = [&](uint8_t* tile) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const __half2 f = __float2half2_rn(fac[v]);
#pragma unroll
        for (int s = 0; s < L::kSlabs; ++s) {
          const uint4 w = raw[s * 4 + v];
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1;
            kv8_to_f16<FMT>(ww[j], a0, a1);
            __half2 x = __hmul2(*reinterpret_cast<__half2*>(&a0), f);
            __half2 y = __hmul2(*reinterpret_cast<__half2*>(&a1), f);
            o[2 * j] = *reinterpret_cast<uint32_t*>(&x);
            o[2 * j + 1] = *reinterpret_cast<uint32_t*>(&y);
          }
          const int row = r4 + 32 * v;
          st_swizzled(tile + s * L::kSlab, row, 2 * cc, make_uint4(o[0], o[1], o[2], o[3]));
          st_swizzled(tile + s * L::kSlab, row, 2 * cc + 1, make_uint4(o[4], o[5], o[6], o[7]));
        }
      }
      fence_async_smem();
      __syncwarp();
    };
    uint32_t good = 0;
    int id = kNone;
    if (nt > 0) {
      place(0, fetch(0));
      load(0);
      good = __ballot_sync(0xffffffffu, grow >= 0) & 0xFFu;
      place(1, fetch(1));
      id = fetch(2);
    }
    for (int i = 0; i < nt; ++i) {
      const int st = i & 1;
      // K's stage is free once Q K^T of tile i - 2 is done with all query tiles;
      // V's once P V of tile i - 2 is, which Q K^T of tile i - 1 came after
      const int after = i - 2 + side;
      if (i >= 2) wait(s_full + 2 * (mts - 1) + (after & 1), (after >> 1) & 1);
      if (!ok) break;
      convert(tiles + st * L::kSlabs * L::kSlab);
      if (warp == 8 && lane == 0) masks[i & 3] = good;
      __syncwarp();
      if (lane == 0) mbar_arrive(side ? kv_full + st : i == 0 ? start : kv_full + (st ^ 1));
      if (i + 1 < nt) {
        load(i + 1);
        good = __ballot_sync(0xffffffffu, grow >= 0) & 0xFFu;
        place(i + 2, id);
        id = fetch(i + 3);
      }
    }
    // There is no K behind the last tile's V, but its arrival is counted: when a
    // tile nt would be converted, so that it cannot fall into an earlier phase.
    if (!side && nt > 0) {
      if (nt >= 2) wait(s_full + 2 * (mts - 1) + (nt & 1), ((nt - 2) >> 1) & 1);
      if (ok && lane == 0) mbar_arrive(kv_full + ((nt - 1) & 1));
    }
  } else {
    // ================================================================ MMA thread
    regs_dec<kRegsMma>();
    if (warp == 16 && lane == 0 && nt > 0) {
    constexpr uint32_t idesc_qk = instr_desc(0, 0, false, false, 128, 128);
    constexpr uint32_t idesc_pv = instr_desc(0, 0, false, true, 128, D);
    const uint64_t kmajor = smem_desc(smem_u32(smem), 16, 1024, 2);
    const uint64_t vmajor = smem_desc(smem_u32(smem), L::kSlab, 1024, 2);
    const uint32_t k_hi = (uint32_t)(kmajor >> 32), v_hi = (uint32_t)(vmajor >> 32);
    const uint32_t qd = (uint32_t)kmajor + L::kQ / 16, kd = (uint32_t)kmajor + L::kK / 16;
    const uint32_t vd = (uint32_t)vmajor + L::kV / 16;
    constexpr uint32_t kTileDesc = L::kSlabs * L::kSlab / 16;
    auto qk = [&](int mt, int st) {
      const uint32_t a = qd + mt * kTileDesc, b2 = kd + st * kTileDesc, d = tmem + 128 * mt;
#pragma unroll
      for (int s = 0; s < L::kSlabs; ++s)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t o = (s * L::kSlab + kk * 32) / 16;
          mma_ss(d, a + o, k_hi, b2 + o, k_hi, idesc_qk, (s | kk) ? 1u : 0u);
        }
    };
    // A wait or a commit takes the issuing thread 200 to 300 cycles while shared
    // memory is busy, and the tensor cores queue few MMAs: so there are three
    // waits and two commits a tile.  MMAs run in order, so S of tile i + 1 also
    // says that P V of tile i is done.
    bool issued = false;
    ok = mbar_wait(start, 0, abort_flag);
    if (ok) {
      tc_fence_after();
      issued = true;
#pragma unroll 1
      for (int mt = 0; mt < mts; ++mt) {
        qk(mt, 0);
        mma_commit(s_full + 2 * mt);
      }
    }
    for (int i = 0; ok && i < nt; ++i) {
      const int st = i & 1, sn = st ^ 1;
      ok = mbar_wait(kv_full + st, (i >> 1) & 1, abort_flag);
#pragma unroll 1
      for (int mt = 0; ok && mt < mts; ++mt) {
        ok = mbar_wait(p_full + mt, i & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + D * mt, tmem + 128 * mt + 8 * kk,
                 vd + st * kTileDesc + kk * 2048 / 16, v_hi, idesc_pv, (i | kk) ? 1u : 0u);
        if (i + 1 == nt) continue;
        qk(mt, sn);
        mma_commit(s_full + 2 * mt + sn);
      }
    }
    if (ok) mma_commit(o_done);
    if (issued) {   // let every issued MMA land before tensor memory is freed
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
    }
  }
  __syncwarp();
  if (!ok) set_status(p.a.status, CSA2_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the key splits of a query row: one warp per row.
template <int D>
__global__ void __launch_bounds__(256) kv8_prefill_combine_kernel(PreParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const Kv8& c = p.a.c;
  const int lane = threadIdx.x & 31, h = blockIdx.y % c.heads, b = blockIdx.y / c.heads;
  const int gr = blockIdx.x * 8 + (threadIdx.x >> 5);
  int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
  ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
  if (gr >= ql * p.a.G) return;
  const int rt = gr / kTileRows, r = gr % kTileRows;
  const int tok = gr / p.a.G, hd = h * p.a.G + gr % p.a.G;
  constexpr int kPer = D / 32;
  float top = -INFINITY, l = 0.0f, o[kPer] = {};
  for (int s = 0; s < p.splits; ++s) {
    const int64_t id =
        (((int64_t)(p.row_tiles - 1 - rt) * c.batch + b) * p.splits + s) * c.heads + h;
    const float* part = p.a.part + id * kTileRows * (D + 2);
    const float m = part[kTileRows * D + r], pl = part[kTileRows * (D + 1) + r];
    if (pl == 0.0f) continue;
    const float nt = fmaxf(top, m);
    const float f = kv8_exp2(top - nt), fm = kv8_exp2(m - nt);
    l = l * f + pl * fm;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + part[r * D + kPer * lane + i] * fm;
    top = nt;
  }
  uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.a.out.data)) + b * p.a.out.sb +
                  tok * p.a.out.st + hd * p.a.out.sh + kPer * lane;
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(out + i) = pack16(o[i] * f, o[i + 1] * f, p.a.out.type);
  if (p.a.lse && lane == 0)
    p.a.lse[((int64_t)b * p.a.T + tok) * p.a.H + hd] =
        l == 0.0f ? -INFINITY : (top + log2f(l) - 7.0f) * 0.6931471805599453f;
}

// left: where the rows outside the cache are joined to the results.
template <int D, int FMT, int KIND>
cudaError_t prefill_as(const PreParams& p, cudaStream_t s, Kv8Left* left) {
  auto kern = kv8_prefill_kernel<D, FMT, KIND>;
  static std::atomic<uint64_t> seen;
  cudaError_t e = kv8_prepare(kern, PreSmem<D>::kBytes, seen);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)p.a.c.heads * p.splits * p.a.c.batch * p.row_tiles;
  e = kv8_launch(kern, dim3((unsigned)grid), kThreads, PreSmem<D>::kBytes, s, p);
  if (left) *left = p.splits == 1 ? Kv8Left{0, 0, 0, 0} : Kv8Left{2, p.row_tiles, kTileRows, p.splits};
  if (e != cudaSuccess || p.splits == 1 || left) return e;
  return kv8_launch(kv8_prefill_combine_kernel<D>,
                    dim3((p.rows + 7) / 8, p.a.c.heads * p.a.c.batch), 256, 0, s, p);
}

template <int KIND>
cudaError_t prefill_any(const Kv8Attn& a, const Kv8Scores& sc, int num_sms, cudaStream_t s,
                        Kv8Left* left) {
  PreParams p{a, a.T * a.G, (a.T * a.G + kTileRows - 1) / kTileRows, 1, sc};
  // Fewer CTAs than SMs: the cached rows are split, into parts of at least 8 tiles.
  const int64_t base = (int64_t)a.c.heads * a.c.batch * p.row_tiles;
  const int limit = num_sms < kKv8SplitCtas ? num_sms : kKv8SplitCtas;
  const int64_t seen = KIND != kPlain ? kv8_most_rows(a, sc) : a.c.max_len;
  if (KIND != kPlain && left) {
    p.splits = kv8_tree_splits(base, seen);
  } else if (2 * base <= limit) {
    const int most = (int)((seen + 8 * kTileKeys - 1) / (8 * kTileKeys));
    p.splits = (int)(limit / base) < most ? (int)(limit / base) : most;
  }
  if (a.c.format == CSA2_KV8_E4M3)
    return a.D == 64 ? prefill_as<64, CSA2_KV8_E4M3, KIND>(p, s, left)
                     : prefill_as<128, CSA2_KV8_E4M3, KIND>(p, s, left);
  return a.D == 64 ? prefill_as<64, CSA2_KV8_INT8, KIND>(p, s, left)
                   : prefill_as<128, CSA2_KV8_INT8, KIND>(p, s, left);
}

}  // namespace
}  // namespace csa2
