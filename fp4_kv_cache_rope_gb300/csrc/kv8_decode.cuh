// Attention over the 8-bit K/V cache for few query rows.
//
//   o_r = sum_j softmax_j(c q_r . k_j) v_j,   k_j = s_K(block) * code,  v_j alike
//
// Few query rows share each cached row (the heads of a group times the tokens
// of the call), so these kernels are bound by the bytes of the cache: 2 D per
// row and head.  The codes go from shared memory into registers, are converted
// there to f16 (exact for both formats) and feed mma.sync with the cached rows
// (then the channels) as M and eight query rows as N, so a group of up to eight
// heads wastes nothing:
//
//   S^T [keys x queries] = K Q^T,   O^T [channels x queries] += V^T P^T
//
// The eight-query tile needs a quarter of that pipe's rate at full HBM
// bandwidth; tcgen05 would want the codes expanded to f16 in shared memory
// first, more shared-memory traffic than the pass has time for.
//
// Exactness.  Queries are scaled per row by a power of two into f16's range
// (the logit factor absorbs it); logits, maxima, sums and outputs are fp32.
// The running maximum is raised when a base-2 logit exceeds it by 8 (a weight of
// 2^8).  The weights P go to f16 for the P V product times 2^7 and times the block's
// V scale over the largest V scale so far: at most 2^15, with f16's full 11 bits
// down to 2^-21; their sum is taken in fp32 before that rounding.
//
// Measured at D 128 and 8 K/V heads, one token a sequence: 32 sequences of up to
// 32768 rows 234 us (6.4 TB/s, 94% of a copy's), 8 of 131072 315 us (6.8 TB/s).
// Few bytes are bound by latency: 5 tokens of 16 sequences of up to 9001 rows, 4
// heads, D 64, 30 us for 8 us of bytes.
//
// Changed scores cost nothing where the bytes bound it: 32 sequences of up to 32768 rows
// with capped scores take 232 us, as without.  With a window a unit's steps are those of
// the rows seen: a token of 8 sequences, window 4096 and 4 first rows, 8 heads, 19 us for
// 67 MB, of which the start, the partial results and their join are a half.
#pragma once

#include "kv8_scores.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 4;                 // of a CTA that shares units with others
constexpr int kThreads = 32 * kWarps;
constexpr int kSub = 32;                  // cached rows of one warp's tile
static_assert(kWarps * kSub == kKv8Step, "a step is one tile per warp");
constexpr int kShort = 2048;              // capacity up to which a unit is one CTA's
constexpr int kShortWarps = 8;

struct DecodeParams {
  Kv8Attn a;
  int32_t rows, tiles;                    // query rows per (sequence, K/V head), tiles of them
  int32_t ctas;
  int32_t row0;                           // first query row (weights)
  Kv8Scores sc;                           // what changes the scores (SCORED)
};

// The cached row of column n (0..7) of an 8-column tile.  Chosen so that the
// 16-byte reads of K (two rows, four chunks each) and of V (four rows, two
// chunks each) by 8 neighbouring lanes fall on different banks of the swizzled
// tile; any order is right as long as the logits and V use the same.
__device__ __forceinline__ int key_of(int n) {
  return (n & 1) ? 2 * ((n >> 1) ^ 2) + 1 : n;
}
// 16-byte chunk position in a tile row, swizzled by the row.
template <int D>
__device__ __forceinline__ int chunk_at(int row, int chunk) {
  return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4)
                  : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src, bool ok) {
  const uint32_t n = ok ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(void* dst, const void* src, bool ok) {
  const uint32_t n = ok ? 4u : 0u;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One query row's 16-bit elements as f16 A fragments: the lane's 16 channels
// of each 64-channel half, scaled by a power of two; returns the logit factor.
// frag[4 half + s][hi]: channels 64 half + 16 t + 4 s + {0,1} (hi 0), + {2,3}.
template <int D>
__device__ __forceinline__ float load_query(const Kv8Rows& q, int64_t at, bool ok, int t,
                                            float scale_log2, uint32_t (&frag)[D / 16][2]) {
  constexpr int kHalf = D / 64;
  uint4 raw[kHalf][2];
  const char* p = static_cast<const char*>(q.data) + 2 * at;
  float amax = 0.0f;
#pragma unroll
  for (int f = 0; f < kHalf; ++f)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      raw[f][u] = make_uint4(0, 0, 0, 0);
      if (ok) raw[f][u] = reinterpret_cast<const uint4*>(p + 128 * f + 32 * t)[u];
    }
  float v[kHalf][16];
#pragma unroll
  for (int f = 0; f < kHalf; ++f) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw[f]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (q.type == CSA2_BF16) {
        bf16x2_to_f32(w[i], v[f][2 * i], v[f][2 * i + 1]);
      } else {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[f][2 * i] = x.x;
        v[f][2 * i + 1] = x.y;
      }
      amax = fmaxf(amax, fmaxf(fabsf(v[f][2 * i]), fabsf(v[f][2 * i + 1])));
    }
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // amax into [2^7, 2^8): exact for every element above 2^-22 of it.  Zero and
  // infinite rows are taken as they are.
  const int e = (int)(__float_as_uint(amax) >> 23);
  const int shift = e == 0 || e == 255 ? 0 : 134 - e;
  const float up = __uint_as_float((uint32_t)(127 + (shift > 127 ? 127 : shift)) << 23);
#pragma unroll
  for (int f = 0; f < kHalf; ++f)
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi)
        frag[4 * f + s][hi] =
            pack16(v[f][4 * s + 2 * hi] * up, v[f][4 * s + 2 * hi + 1] * up, CSA2_F16);
  return scale_log2 / up;
}

// 8x8 matrix of 16-bit elements, row lane / 4, columns 2 (lane % 4) + {0, 1}:
// its transpose in the same layout.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int WARPS>
struct DecodeSmem {
  static constexpr int kStages = 3;
  static constexpr int kTile = kSub * D;                 // bytes of K (and of V) per stage
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRingWarp = kStages * kStage;
  static constexpr int kMeta = WARPS * kRingWarp;        // per warp and stage: 4 scales, 2 flags
  static constexpr int kMetaWarp = kStages * 32;
  static constexpr int kStat = kMeta + WARPS * kMetaWarp;   // m, l: fp32 [WARPS][32] each
  static constexpr int kBytes = kStat + 2 * WARPS * 32 * 4;
  static constexpr int kRedRow = D + 4;                  // merge buffer (over the ring)
  static constexpr bool fits(int nt) { return WARPS * 8 * nt * kRedRow * 4 <= kMeta; }
};

// Where a unit's partial result of CTA i goes: slot 2 i when the unit began in
// an earlier CTA, 2 i + 1 when it begins in CTA i and ends in a later one.
__host__ __device__ constexpr int64_t slot_floats(int D) { return kKv8SlotRows * (D + 2); }

// The two 16-row groups of a warp's tile of cached rows.
struct Groups {
  int64_t row[2];   // row index of the group's first row, -1: none
  int64_t blk[2];   // index of its scale
};
constexpr int kNoRows = -0x7FFFFFFF - 1;
// A warp stops at the first use of a value that is still on its way, so the page
// ids are read a tile before they are used.  Lane parity does one group each.
__device__ __forceinline__ int fetch_page(const Kv8& c, int b, int pos, int n, int lane) {
  const int mine = pos + 16 * (lane & 1);
  return mine < n ? kv8_page_id(c, b, mine) : kNoRows;
}
__device__ __forceinline__ Groups place_groups(const Kv8& c, int id, int h, int pos,
                                               uint32_t* status, int lane) {
  int64_t row = -1, blk = 0;
  if (id != kNoRows) {
    int in_page;
    kv8_in_page(c, pos + 16 * (lane & 1), in_page);
    const int page = kv8_check(c, id);
    if (page >= 0) {
      row = kv8_row(c, page, h, in_page);
      blk = kv8_block(c, page, h, in_page);
    } else if (lane < 2) {
      set_status(status, CSA2_DEV_BAD_PAGE);
    }
  }
  Groups g;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    g.row[u] = __shfl_sync(0xffffffffu, row, u);
    g.blk[u] = __shfl_sync(0xffffffffu, blk, u);
  }
  return g;
}

// CTAs that an SM holds: by the shared memory, and by the registers that more
// query rows take.
constexpr int decode_ctas(int D, int nt, int warps) {
  return warps != kWarps ? 1 : D == 128 ? 2 : nt == 1 ? 4 : 3;
}

// NT: tiles of eight query rows.  WARPS = kWarps: the steps of all units are
// shared out evenly; kShortWarps: every unit is one CTA's, and no partial results
// are left to join.  SCORED: p.sc changes the scores and which rows count; a unit's
// steps are then those of the rows that any of its sequence's queries sees.
template <int D, int NT, int FMT, int WARPS, bool SCORED>
__global__ void __launch_bounds__(32 * WARPS, decode_ctas(D, NT, WARPS))
    kv8_decode_kernel(DecodeParams p) {
  using L = DecodeSmem<D, WARPS>;
  static_assert(L::fits(NT), "merge buffer");
  constexpr bool kWhole = WARPS != kWarps;
  constexpr int kStep = WARPS * kSub;
  constexpr int kHalf = D / 64;
  constexpr int kMT = D / 16;                // 16-channel tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const Kv8& c = p.a.c;
  griddep_wait();
  griddep_launch_dependents();

  uint8_t* ring = smem + warp * L::kRingWarp;
  uint8_t* meta = smem + L::kMeta + warp * L::kMetaWarp;
  float* sm = reinterpret_cast<float*>(smem + L::kStat);
  float* sl = sm + WARPS * 32;

  const int units = c.heads * p.tiles;
  int b, n, steps, unit, st0;
  int64_t x = 0, x1 = 0;
  Kv8Span span{};                          // SCORED: the steps' rows
  if (kWhole) {
    b = blockIdx.x / units;
    unit = blockIdx.x % units;
    n = kv8_len(c, b);
    steps = n <= kStep ? 1 : (n + kStep - 1) / kStep;
    if (SCORED) {
      span = kv8_span<kStep>(p.a, p.sc, b);
      steps = span.steps;
    }
    st0 = 0;
    x1 = steps;
  } else if (SCORED) {
    const Kv8SpanShare at = kv8_share_by(c, lane, units, p.ctas, blockIdx.x, [&](int i) {
      return kv8_span<kStep>(p.a, p.sc, i);
    });
    if ((int)blockIdx.x >= at.ctas) return;
    x = at.x;
    x1 = at.x1;
    b = at.b;
    span = at.span;
    n = at.n;
    steps = at.steps;
    unit = at.unit;
    st0 = at.step;
  } else {
    const Kv8Share at = kv8_share(c, lane, units, p.ctas, blockIdx.x);
    if ((int)blockIdx.x >= at.ctas) return;
    x = at.x;
    x1 = at.x1;
    b = at.b;
    n = at.n;
    steps = at.steps;
    unit = at.unit;
    st0 = at.step;
  }

  // this lane's places in a stage: 16-byte chunk `lane + 32 i` of the tile's
  // codes goes to dst[i & 1] + 512 i (D 128; rows of 64 bytes: dst[0] + 512 i)
  const int dst0 = chunk_at<D>(lane * 16 / D, lane % (D / 16));
  const int dst1 = D == 128 ? chunk_at<D>(lane * 16 / D + 4, lane % (D / 16)) - 512 : dst0;

  // first row of this warp's tile of step st
  auto row_of = [&](int st) {
    return (SCORED ? span.row(st, kStep) : st * kStep) + warp * kSub;
  };

  while (x < x1) {
    const int st1 = (int)min((int64_t)steps, st0 + (x1 - x));
    const int h = unit / p.tiles, row0 = (unit % p.tiles) * 8 * NT;
    int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
    ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);

    // ---- pipeline over this warp's tiles st0 .. st1
    Groups next;
    int id;
    auto fetch = [&](int st) {
      id = fetch_page(c, b, row_of(st), st < st1 ? n : 0, lane);
    };
    auto place = [&](int st) {
      next = place_groups(c, id, h, row_of(st), p.a.status, lane);
    };
    auto issue = [&](int st, int stage) {
      if (st < st1) {
        const int left = n - row_of(st);
        uint8_t* k = ring + stage * L::kStage;
        const int64_t at[2] = {next.row[0] * D + lane * 16, next.row[1] * D + lane * 16};
        if (left >= kSub && next.row[0] >= 0 && next.row[1] >= 0) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int64_t off = at[i / (D / 32)] + 512 * (i % (D / 32));
            uint8_t* to = k + (i & 1 ? dst1 : dst0) + 512 * i;
            cp_async16(to, c.codes[0] + off);
            cp_async16(to + L::kTile, c.codes[1] + off);
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const bool ok = next.row[i / (D / 32)] >= 0 && (lane + 32 * i) * 16 / D < left;
            const int64_t off = ok ? at[i / (D / 32)] + 512 * (i % (D / 32)) : 0;
            uint8_t* to = k + (i & 1 ? dst1 : dst0) + 512 * i;
            cp_async16_zfill(to, c.codes[0] + off, ok);
            cp_async16_zfill(to + L::kTile, c.codes[1] + off, ok);
          }
        }
        float* m = reinterpret_cast<float*>(meta + stage * 32);
        const bool ok = (lane & 1 ? next.row[1] : next.row[0]) >= 0;
        const int64_t sc = lane & 1 ? next.blk[1] : next.blk[0];
        if (lane < 4) cp_async4_zfill(m + lane, c.scales[lane >> 1] + (ok ? sc : 0), ok);
        if (lane < 2) reinterpret_cast<int*>(m)[4 + lane] = ok;
      }
      cp_async_commit();
    };
    fetch(st0);
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) {
      place(st0 + i);
      fetch(st0 + i + 1);
      issue(st0 + i, i);
    }

    // ---- queries of this unit: row 8 u + g as B fragments; the logit factor
    // and the number of visible cached rows of the rows 8 u + 2 t + e
    uint32_t qf[NT][D / 16][2];
    float mul[NT][2];
    int lim[NT][2], full = 0x7FFFFFFF;   // rows below `full` are seen by every query row
    // SCORED: lim is the query's position; the slope in base 2; rows below `low` may
    // be in front of a window
    float slope[NT][2];
    int low = 0, prefix = 0;
    if (SCORED) prefix = p.sc.prefix ? p.sc.prefix[b] : 0;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int row = row0 + 8 * u + g;
      const int tok = row / p.a.G, hd = h * p.a.G + row % p.a.G;
      const bool ok = row < p.rows && tok < ql;
      const float f = load_query<D>(p.a.q, b * p.a.q.sb + tok * p.a.q.st + hd * p.a.q.sh, ok, t,
                                    SCORED ? p.sc.factor : p.a.scale_log2, qf[u]);
      // a row without a query is never written: it may see everything
      int see = ok ? min(n, n - ql + tok + 1) : 0x7FFFFFFF;
      float sl = 0.0f;
      if (SCORED) {
        see = ok ? kv8_query_at(p.a, p.sc, b, n, ql, tok) : kNoQuery;
        if (ok) {
          full = min(full, p.sc.sees(see, n, prefix));
          low = max(low, p.sc.from(see));
          if (p.sc.slopes) sl = p.sc.slopes[hd] * kLog2e;
        }
      } else {
        full = min(full, see);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mul[u][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + e));
        lim[u][e] = __shfl_sync(0xffffffffu, see, 4 * (2 * t + e));
        slope[u][e] = SCORED ? __shfl_sync(0xffffffffu, sl, 4 * (2 * t + e)) : 0.0f;
      }
    }
    full = __reduce_min_sync(0xffffffffu, full);
    if (SCORED) low = __reduce_max_sync(0xffffffffu, low);

    float o[NT][kMT][4];
    float mx[NT][2], ls[NT][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int j = 0; j < kMT; ++j) o[u][j][0] = o[u][j][1] = o[u][j][2] = o[u][j][3] = 0.0f;
      mx[u][0] = mx[u][1] = -INFINITY;
      ls[u][0] = ls[u][1] = 0.0f;
    }
    float vref = 0.0f;     // the largest V scale so far (a power of two)

    int stage = 0;
    for (int st = st0; st < st1; ++st) {
      cp_async_wait<L::kStages - 2>();
      __syncwarp();
      {
        const int nxt = st + L::kStages - 1;
        place(nxt);
        fetch(nxt + 1);
        issue(nxt, stage == 0 ? L::kStages - 1 : stage - 1);
      }
      const uint8_t* k = ring + stage * L::kStage;
      const uint8_t* v = k + L::kTile;
      const float4 sc = *reinterpret_cast<const float4*>(meta + stage * 32);
      const int2 there = *reinterpret_cast<const int2*>(meta + stage * 32 + 16);
      const float ks[2] = {sc.x, sc.y}, vs[2] = {sc.z, sc.w};
      stage = stage + 1 == L::kStages ? 0 : stage + 1;

      // ---- S^T = K Q^T: two tiles of 16 cached rows (rows key_of(g), + 8)
      float s[NT][2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int u = 0; u < NT; ++u) s[u][i][0] = s[u][i][1] = s[u][i][2] = s[u][i][3] = 0.0f;
        const int row = 16 * i + key_of(g);
#pragma unroll
        for (int f = 0; f < kHalf; ++f) {
          const uint4 wa = *reinterpret_cast<const uint4*>(k + chunk_at<D>(row, 4 * f + t));
          const uint4 wb = *reinterpret_cast<const uint4*>(k + chunk_at<D>(row + 8, 4 * f + t));
          const uint32_t xa[4] = {wa.x, wa.y, wa.z, wa.w}, xb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t a[4];
            kv8_to_f16<FMT>(xa[q], a[0], a[2]);
            kv8_to_f16<FMT>(xb[q], a[1], a[3]);
#pragma unroll
            for (int u = 0; u < NT; ++u) mma16816(s[u][i], a, qf[u][4 * f + q][0], qf[u][4 * f + q][1]);
          }
        }
      }

      // ---- logits (base 2): s[u][i][2 r + e] is cached row 16 i + 8 r + key_of(g),
      // query row 8 u + 2 t + e
      const int pos = row_of(st);
      bool raise = false;
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) s[u][i][2 * r + e] *= mul[u][e] * ks[i];
      if (SCORED) {
        if (p.sc.cap2 > 0.0f) {
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[u][i][e] = kv8_cap(s[u][i][e], p.sc.cap2);
        }
        if (p.sc.slopes) {
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const float d = (float)(lim[u][e] - (pos + 16 * i + 8 * r + key_of(g)));
                  s[u][i][2 * r + e] = fmaf(-slope[u][e], fabsf(d), s[u][i][2 * r + e]);
                }
        }
        if (pos + kSub > full || (pos < low && pos + kSub > p.sc.sink) || !(there.x & there.y)) {
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int to = min(p.sc.sees(lim[u][e], n, prefix), n), from = p.sc.from(lim[u][e]);
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const int j = pos + 16 * i + 8 * r + key_of(g);
                  if (j >= to || (j < from && j >= p.sc.sink) || !(i ? there.y : there.x))
                    s[u][i][2 * r + e] = -INFINITY;
                }
            }
        }
      } else if (pos + kSub > full || !(there.x & there.y)) {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (pos + 16 * i + 8 * r + key_of(g) >= min(lim[u][e], n) ||
                    !(i ? there.y : there.x))
                  s[u][i][2 * r + e] = -INFINITY;
      }
      float tops[NT][2];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tops[u][e] = fmaxf(fmaxf(s[u][0][e], s[u][0][2 + e]), fmaxf(s[u][1][e], s[u][1][2 + e]));
          raise |= tops[u][e] > mx[u][e] + 8.0f;
        }
      const float vnew = fmaxf(vref, fmaxf(vs[0], vs[1]));
      if (__any_sync(0xffffffffu, raise) || vnew > vref) {
        // raise the maxima and the V reference; O and the sums follow
        const float vdown = vnew > vref ? vref * kv8_inverse(vnew) : 1.0f;
        vref = vnew;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = tops[u][e];
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = fmaxf(top, mx[u][e]);
            alpha[e] = top == -INFINITY ? 1.0f : kv8_exp2(mx[u][e] - top);
            mx[u][e] = top;
            ls[u][e] *= alpha[e];
            alpha[e] *= vdown;
          }
#pragma unroll
          for (int j = 0; j < kMT; ++j) {
            o[u][j][0] *= alpha[0];
            o[u][j][1] *= alpha[1];
            o[u][j][2] *= alpha[0];
            o[u][j][3] *= alpha[1];
          }
        }
      }
      // ---- P^T in f16, transposed into the B fragments of the P V product
      const float vinv = kv8_inverse(vref);
      const float vr[2] = {vs[0] * vinv * 128.0f, vs[1] * vinv * 128.0f};
      uint32_t pf[NT][2][2];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const float use[2] = {mx[u][0] == -INFINITY ? 0.0f : mx[u][0],
                              mx[u][1] == -INFINITY ? 0.0f : mx[u][1]};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float wa = kv8_exp2(s[u][i][2 * r] - use[0]);
            const float wb = kv8_exp2(s[u][i][2 * r + 1] - use[1]);
            ls[u][0] += wa;
            ls[u][1] += wb;
            pf[u][i][r] = transpose8x8(pack16(wa * vr[i], wb * vr[i], CSA2_F16));
          }
      }

      // ---- O^T += V^T P^T: rows g, g + 8 of output tile j are the channels
      // (D/8) g + 2 j and + 1, its columns the query rows
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[4][D / 32];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int row = 16 * i + 8 * (y >> 1) + key_of(2 * t + (y & 1));
          if (D == 128) {
            const uint4 z = *reinterpret_cast<const uint4*>(v + chunk_at<D>(row, g));
            w[y][0] = z.x; w[y][1] = z.y; w[y][D / 32 - 2] = z.z; w[y][D / 32 - 1] = z.w;
          } else {
            const uint2 z =
                *reinterpret_cast<const uint2*>(v + chunk_at<D>(row, g >> 1) + 8 * (g & 1));
            w[y][0] = z.x; w[y][1] = z.y;
          }
        }
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t a[4], d[4];
          kv8_to_f16<FMT>(__byte_perm(w[0][q], w[1][q], 0x5140), a[0], a[1]);
          kv8_to_f16<FMT>(__byte_perm(w[2][q], w[3][q], 0x5140), a[2], a[3]);
          kv8_to_f16<FMT>(__byte_perm(w[0][q], w[1][q], 0x7362), d[0], d[1]);
          kv8_to_f16<FMT>(__byte_perm(w[2][q], w[3][q], 0x7362), d[2], d[3]);
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            mma16816(o[u][2 * q], a, pf[u][i][0], pf[u][i][1]);
            mma16816(o[u][2 * q + 1], d, pf[u][i][0], pf[u][i][1]);
          }
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();

    // ---- merge the warps (over the ring), then write the rows or a partial result
    const bool whole = kWhole || (st0 == 0 && st1 == steps);
    float* part = p.a.part + (2 * (int64_t)blockIdx.x + (st0 > 0 ? 0 : 1)) * slot_floats(D);
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ls[u][e] += __shfl_xor_sync(0xffffffffu, ls[u][e], 4);
        ls[u][e] += __shfl_xor_sync(0xffffffffu, ls[u][e], 8);
        ls[u][e] += __shfl_xor_sync(0xffffffffu, ls[u][e], 16);
        if (g == 0) {
          sm[warp * 32 + 8 * u + 2 * t + e] = mx[u][e];
          sl[warp * 32 + 8 * u + 2 * t + e] = ls[u][e];
        }
      }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * u + 2 * t + e;
        float top = sm[row];
#pragma unroll
        for (int i = 1; i < WARPS; ++i) top = fmaxf(top, sm[i * 32 + row]);
        // a sum of 0: no row was visible; of NaN: the query holds one
        const float f = ls[u][e] == 0.0f ? 0.0f : kv8_exp2(mx[u][e] - top) * (vref * 0x1p-7f);
        float* to = red + (warp * 8 * NT + row) * L::kRedRow + (D / 8) * g;
#pragma unroll
        for (int j = 0; j < kMT; j += 2)
          *reinterpret_cast<float4*>(to + 2 * j) =
              make_float4(o[u][j][e] * f, o[u][j][2 + e] * f, o[u][j + 1][e] * f,
                          o[u][j + 1][2 + e] * f);
      }
    __syncthreads();
    // 8 channels a thread
    for (int at = tid; at < 8 * NT * (D / 8); at += 32 * WARPS) {
      const int row = at / (D / 8), ch = 8 * (at % (D / 8));
      float top = sm[row], l = 0.0f;
#pragma unroll
      for (int i = 1; i < WARPS; ++i) top = fmaxf(top, sm[i * 32 + row]);
      float y[8] = {};
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        const float wl = sl[i * 32 + row];
        l += wl == 0.0f ? 0.0f : wl * kv8_exp2(sm[i * 32 + row] - top);
        const float4* from =
            reinterpret_cast<const float4*>(red + (i * 8 * NT + row) * L::kRedRow + ch);
        const float4 ya = from[0], yb = from[1];
        y[0] += ya.x; y[1] += ya.y; y[2] += ya.z; y[3] += ya.w;
        y[4] += yb.x; y[5] += yb.y; y[6] += yb.z; y[7] += yb.w;
      }
      const int gr = row0 + row, tok = gr / p.a.G, hd = h * p.a.G + gr % p.a.G;
      if (gr >= p.rows || tok >= ql) continue;
      if (SCORED && whole && p.sc.rows_out) {   // the drafted rows are still to come
        float* to = p.sc.rows_out + (((int64_t)b * p.a.T + tok) * p.a.H + hd) * kv8_row_floats(D);
        *reinterpret_cast<float4*>(to + ch) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(to + ch + 4) = make_float4(y[4], y[5], y[6], y[7]);
        if (ch == 0) {
          to[D] = top;
          to[D + 1] = l;
        }
      } else if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.a.out.data)) + b * p.a.out.sb +
                        tok * p.a.out.st + hd * p.a.out.sh + ch;
        *reinterpret_cast<uint4*>(out) = make_uint4(
            pack16(y[0] * inv, y[1] * inv, p.a.out.type), pack16(y[2] * inv, y[3] * inv, p.a.out.type),
            pack16(y[4] * inv, y[5] * inv, p.a.out.type), pack16(y[6] * inv, y[7] * inv, p.a.out.type));
        if (p.a.lse && ch == 0)
          p.a.lse[((int64_t)b * p.a.T + tok) * p.a.H + hd] =
              l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
      } else {
        float4* po = reinterpret_cast<float4*>(part + row * D + ch);
        po[0] = make_float4(y[0], y[1], y[2], y[3]);
        po[1] = make_float4(y[4], y[5], y[6], y[7]);
        if (ch == 0) {
          part[kKv8SlotRows * D + row] = top;
          part[kKv8SlotRows * (D + 1) + row] = l;
        }
      }
    }
    if (kWhole) return;
    __syncthreads();   // the ring takes the next unit's rows

    // ---- next unit
    x += st1 - st0;
    st0 = 0;
    if (st1 == steps && ++unit == units && x < x1) {
      unit = 0;
      ++b;
      if (SCORED) {
        span = kv8_span<kStep>(p.a, p.sc, b);
        n = span.n;
        steps = span.steps;
      } else {
        n = kv8_len(c, b);
        steps = kv8_steps(c, b);
      }
    }
  }
}

// Joins the partial results of the units that several CTAs shared: one CTA per
// query row of a unit, four channels a thread, its threads' groups taking every
// kCombine-th part.  The order of the sums is fixed by the split.
constexpr int kCombine = 4;
template <int D, bool SCORED>
__global__ void __launch_bounds__(D / 4 * kCombine) kv8_combine_kernel(DecodeParams p, int tile_rows) {
  griddep_wait();
  griddep_launch_dependents();
  const Kv8& c = p.a.c;
  const int tid = threadIdx.x, lane = tid & 31;
  const int units = c.heads * p.tiles;
  const int b = blockIdx.x / units, unit = blockIdx.x % units, row = blockIdx.y;
  const int h = unit / p.tiles, gr = (unit % p.tiles) * tile_rows + row;
  const int tok = gr / p.a.G, hd = h * p.a.G + gr % p.a.G;
  int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
  ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
  if (gr >= p.rows || tok >= ql) return;
  int c0, c1;
  if (SCORED)
    kv8_sharers_by(c, lane, units, p.ctas, b, unit, c0, c1,
                   [&](int i) { return kv8_span<kKv8Step>(p.a, p.sc, i).steps; });
  else
    kv8_sharers_of(c, lane, units, p.ctas, b, unit, c0, c1);
  if (c0 == c1) return;
  // the unit began in CTA c0's second slot and went on in the others' first; each
  // group joins its parts as they come, then the groups are joined
  __shared__ float tops[kCombine], sums[kCombine];
  __shared__ float4 outs[kCombine][D / 4];
  const int parts = c1 - c0 + 1;
  const int grp = tid / (D / 4), ch = tid % (D / 4);
  float top = -INFINITY, l = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  auto join = [&](float m, float pl, const float4& y) {
    const float nt = fmaxf(top, m);
    // a sum of 0: the part saw no row; of NaN: the query holds one, and it stays
    const float f = l == 0.0f ? 0.0f : kv8_exp2(top - nt), g = pl == 0.0f ? 0.0f : kv8_exp2(m - nt);
    l = l * f + pl * g;
    o.x = o.x * f + y.x * g;
    o.y = o.y * f + y.y * g;
    o.z = o.z * f + y.z * g;
    o.w = o.w * f + y.w * g;
    top = nt;
  };
#pragma unroll 4
  for (int i = grp; i < parts; i += kCombine) {
    const float* part = p.a.part + (2 * (int64_t)(c0 + i) + (i == 0)) * slot_floats(D);
    join(part[kKv8SlotRows * D + row], part[kKv8SlotRows * (D + 1) + row],
         reinterpret_cast<const float4*>(part + row * D)[ch]);
  }
  if (ch == 0) {
    tops[grp] = top;
    sums[grp] = l;
  }
  outs[grp][ch] = o;
  __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int k = 1; k < kCombine; ++k) join(tops[k], sums[k], outs[k][ch]);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.a.out.data)) + b * p.a.out.sb +
                  tok * p.a.out.st + hd * p.a.out.sh + 4 * ch;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack16(o.x * inv, o.y * inv, p.a.out.type),
                                              pack16(o.z * inv, o.w * inv, p.a.out.type));
  if (p.a.lse && tid == 0)
    p.a.lse[((int64_t)b * p.a.T + tok) * p.a.H + hd] =
        l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

// left: the way the rows outside the cache have to take from here (the split).
template <int D, int NT, int FMT, bool SCORED>
cudaError_t decode_as(DecodeParams p, int num_sms, cudaStream_t s, Kv8Left* left) {
  const int64_t units = (int64_t)p.a.c.batch * p.a.c.heads * p.tiles;
  // Short caches in one launch: 1000 rows take as long on the GPU as shared out
  // and joined (10.5 us), 2000 rows of few units longer (14.5 us against 10.4 us),
  // and the host, which bounds such calls, issues one launch less.
  // (Drafted tokens' results are joined with their rows anyway: few units are shared.)
  if ((SCORED ? kv8_most_rows(p.a, p.sc) : p.a.c.max_len) <= kShort && !(left && units < num_sms)) {
    using L = DecodeSmem<D, kShortWarps>;
    auto kern = kv8_decode_kernel<D, NT, FMT, kShortWarps, SCORED>;
    static std::atomic<uint64_t> seen;
    const cudaError_t e = kv8_prepare(kern, L::kBytes, seen);
    if (e != cudaSuccess) return e;
    return kv8_launch(kern, dim3((unsigned)units), 32 * kShortWarps, L::kBytes, s, p);
  }
  using L = DecodeSmem<D, kWarps>;
  auto kern = kv8_decode_kernel<D, NT, FMT, kWarps, SCORED>;
  static std::atomic<uint64_t> seen;
  cudaError_t e = kv8_prepare(kern, L::kBytes, seen);
  if (e != cudaSuccess) return e;
  const int ctas = decode_ctas(D, NT, kWarps) * num_sms;
  p.ctas = ctas < kKv8Ctas ? ctas : kKv8Ctas;
  e = kv8_launch(kern, dim3(p.ctas), kThreads, L::kBytes, s, p);
  if (left) *left = Kv8Left{1, p.tiles, 8 * NT, p.ctas};
  if (e != cudaSuccess || left) return e;
  return kv8_launch(kv8_combine_kernel<D, SCORED>, dim3((unsigned)units, 8 * NT), D / 4 * kCombine, 0, s, p,
                    8 * NT);
}
template <int D, int FMT, bool SCORED>
cudaError_t decode_of(DecodeParams p, int num_sms, cudaStream_t s, Kv8Left* left = nullptr) {
  // More than 24 rows go as several tiles of 16, whose cached rows come from L2
  // the second time: 16 sequences of 9000 rows, 32 query rows, D 128: 47 us
  // against 70 us in one tile of 32, which does not fit the registers.
  const int nt = p.rows <= 8 ? 1 : p.rows <= 16 || p.rows > 24 ? 2 : 3;
  p.tiles = (p.rows + 8 * nt - 1) / (8 * nt);
  return nt == 1   ? decode_as<D, 1, FMT, SCORED>(p, num_sms, s, left)
         : nt == 2 ? decode_as<D, 2, FMT, SCORED>(p, num_sms, s, left)
                   : decode_as<D, 3, FMT, SCORED>(p, num_sms, s, left);
}
}  // namespace
}  // namespace csa2
