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
// 2^15, with f16's full precision down to 2^-21.  l is summed in fp32 from the
// unrounded weights.
//
// Warps (640 threads): 0-3 and 4-7 softmax of query tile 0 and 1; 8-11 turn K's
// codes into f16 tiles and 12-15 V's, from registers loaded one tile ahead (no
// raw copy in shared memory, whose bandwidth the MMAs need); 16 issues the MMAs.
//
// A softmax thread reads its row's 128 logits from tensor memory twice, 16 at a
// time with the next ones on their way: once for the maximum, once for the
// exponentials.  That
// keeps every role within its registers: a spilled register is read back from
// L2, because L1 is left little beside the tiles.
#include "kv8_mma.cuh"

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

struct PreParams {
  Kv8Attn a;
  int32_t rows, row_tiles, splits;
};

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefill_kernel(PreParams p) {
  using L = PreSmem<D>;
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
  const int keys = max(0, min(n, n - ql + last_tok + 1));
  const int all_tiles = (keys + kTileKeys - 1) / kTileKeys;
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
    const int lim = real ? min(n, n - ql + tok + 1) : 0x7FFFFFFF;
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
      mul = p.a.scale_log2 / up;               // times K's largest scale, below
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
      const int key0 = (t0 + i) * kTileKeys;
      const bool masked = groups != 0xFFu || __any_sync(0xffffffffu, lim < key0 + kTileKeys);
      const int seen = masked ? (int)__reduce_min_sync(0xffffffffu, max(lim - key0, 0)) : 0;
      auto hide = [&](uint32_t (&s)[16], int u) {          // columns 16 u ..
        const bool gone = !((groups >> u) & 1u);
        if (!gone && seen >= 16 * u + 16) return;          // every row sees them
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (gone || key0 + 16 * u + j >= lim) s[j] = 0xFF800000u;
      };
      // f(columns 16 u .., u) for u = 0 .. 7, the next ones on their way meanwhile
      auto each = [&](auto f) {
        uint32_t sa[16], sb[16];
        tmem_ld16(tS, sa);
        tmem_ld_wait();
        reg_fence(sa);
#pragma unroll
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
      float tops[2] = {-INFINITY, -INFINITY};
      auto largest = [&](uint32_t (&s)[16], int) {
#pragma unroll
        for (int j = 0; j < 16; j += 2)
          tops[(j >> 1) & 1] =
              fmaxf(tops[(j >> 1) & 1], fmaxf(__uint_as_float(s[j]), __uint_as_float(s[j + 1])));
      };
      if (masked) {
        each([&](uint32_t (&s)[16], int u) {
          hide(s, u);
          largest(s, u);
        });
      } else {
        each(largest);
      }
      const float top = fmaxf(tops[0], tops[1]) * mul;
      // (a row without a visible key so far waits for one; no row's result
      // depends on another's)
      const bool raise = top > m + 8.0f;
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
      const float mm = m == -INFINITY ? 0.0f : m;
      const uint64_t f2 = pack2(mul, mul), u2 = pack2(7.0f - mm, 7.0f - mm);
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
      if (__any_sync(0xffffffffu, fabsf(mm) > 65536.0f)) {
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
          uint32_t s[16];
          tmem_ld16(tS + 16 * u, s);
          tmem_ld_wait();
          reg_fence(s);
          hide(s, u);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            s[j] = __float_as_uint((__fmul_rn(__uint_as_float(s[j]), mul) - mm) + 7.0f);
          weights(s, u);
        }
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
    if (p.splits == 1) {
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
#pragma unroll 4
      for (int pos = t0 * kTileKeys / blk * blk + ct * blk; pos < end; pos += 128 * blk) {
        int in_page;
        const int page = kv8_page(c, b, pos, in_page);
        if (page >= 0) mx = fmaxf(mx, scales[kv8_block(c, page, h, in_page)]);
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
      const int pos = (t0 + i) * kTileKeys + 16 * (lane & 7);
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
        kv8_in_page(c, (t0 + i) * kTileKeys + 16 * (lane & 7), in_page);
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
        const bool in = g >= 0 && (t0 + i) * kTileKeys + row < keys;
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

template <int D, int FMT>
cudaError_t prefill_as(const PreParams& p, cudaStream_t s) {
  auto kern = kv8_prefill_kernel<D, FMT>;
  static std::atomic<uint64_t> seen;
  cudaError_t e = kv8_prepare(kern, PreSmem<D>::kBytes, seen);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)p.a.c.heads * p.splits * p.a.c.batch * p.row_tiles;
  e = kv8_launch(kern, dim3((unsigned)grid), kThreads, PreSmem<D>::kBytes, s, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return kv8_launch(kv8_prefill_combine_kernel<D>,
                    dim3((p.rows + 7) / 8, p.a.c.heads * p.a.c.batch), 256, 0, s, p);
}

}  // namespace

size_t kv8_prefill_part_bytes(int D) { return (size_t)kKv8SplitCtas * kTileRows * (D + 2) * 4; }

cudaError_t launch_kv8_prefill(const Kv8Attn& a, int num_sms, cudaStream_t s) {
  PreParams p{a, a.T * a.G, (a.T * a.G + kTileRows - 1) / kTileRows, 1};
  // Fewer CTAs than SMs: the cached rows are split, into parts of at least 8 tiles.
  const int64_t base = (int64_t)a.c.heads * a.c.batch * p.row_tiles;
  const int limit = num_sms < kKv8SplitCtas ? num_sms : kKv8SplitCtas;
  if (2 * base <= limit) {
    const int most = (a.c.max_len + 8 * kTileKeys - 1) / (8 * kTileKeys);
    p.splits = (int)(limit / base) < most ? (int)(limit / base) : most;
  }
  if (a.c.format == CSA2_KV8_E4M3)
    return a.D == 64 ? prefill_as<64, CSA2_KV8_E4M3>(p, s) : prefill_as<128, CSA2_KV8_E4M3>(p, s);
  return a.D == 64 ? prefill_as<64, CSA2_KV8_INT8>(p, s) : prefill_as<128, CSA2_KV8_INT8>(p, s);
}

cudaError_t set_wait_limit_kv8_prefill(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace csa2
