// Attention over the 8-bit K/V cache for few query rows, and the weights that
// each cached row gets.
//
//   o_r = sum_j softmax_j(c q_r . k_j) v_j,   k_j = s_K(block) * code,  v_j alike
//
// Few query rows share each cached row (the heads of a group times the tokens
// of the call), so these kernels are bound by the bytes of the cache: 2 D per
// row and head.  The codes go from shared memory into registers, are converted
// there to f16 (exact for both formats) and feed mma.sync; a 16-row tile of
// queries then needs well under half of that pipe's rate at full HBM bandwidth
// (tcgen05 would need the codes expanded to f16 in shared memory first, which
// costs more shared-memory bandwidth than the pass has).
//
// Exactness.  Queries are scaled per row by a power of two into f16's range
// (the logit factor absorbs it); logits, maxima, sums and outputs are fp32.
// The weights P go to f16 for the P V product times 2^15 and times the block's
// V scale over the largest V scale so far: a weight keeps f16's 11 bits down to
// 2^-29 of the largest weight, and the sum of the weights is taken in fp32
// before that rounding.
#include "kv8.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSub = 32;                  // cached rows of one warp's tile
static_assert(kWarps * kSub == kKv8Step, "a step is one tile per warp");

struct DecodeParams {
  Kv8Attn a;
  int32_t rows, tiles;                    // query rows per (sequence, K/V head), tiles of them
  int32_t ctas;
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

template <int D>
struct DecodeSmem {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kTile = kSub * D;                 // bytes of K (and of V) per stage
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRingWarp = kStages * kStage;
  static constexpr int kMeta = kWarps * kRingWarp;       // per warp and stage: 4 scales, 2 flags
  static constexpr int kMetaWarp = kStages * 32;
  static constexpr int kRed = kMeta + kWarps * kMetaWarp;  // fp32 [16][D + 4] merge buffer
  static constexpr int kStat = kRed + 16 * (D + 4) * 4;    // m, l: fp32 [kWarps][32] each
  static constexpr int kBytes = kStat + 2 * kWarps * 32 * 4;
};

// Where a unit's partial result of CTA i goes: slot 2 i when the unit began in
// an earlier CTA, 2 i + 1 when it begins in CTA i and ends in a later one.
__host__ __device__ constexpr int64_t slot_floats(int D) { return kKv8SlotRows * (D + 2); }

template <int D, int MT, int FMT>
__global__ void __launch_bounds__(kThreads, 2) kv8_decode_kernel(DecodeParams p) {
  using L = DecodeSmem<D>;
  constexpr int kChunks = D / 16;
  constexpr int kNT = D / 8;                 // 8-channel tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const Kv8& c = p.a.c;
  griddep_wait();
  griddep_launch_dependents();

  uint8_t* ring = smem + warp * L::kRingWarp;
  uint8_t* meta = smem + L::kMeta + warp * L::kMetaWarp;
  float* red = reinterpret_cast<float*>(smem + L::kRed);
  float* sm = reinterpret_cast<float*>(smem + L::kStat);
  float* sl = sm + kWarps * 32;

  const int units = c.heads * p.tiles;
  const int64_t total = kv8_total(c, lane) * units;
  const int ctas = kv8_sharers(total, p.ctas);
  if ((int)blockIdx.x >= ctas) return;
  int64_t x = total * blockIdx.x / ctas;
  const int64_t x1 = total * (blockIdx.x + 1) / ctas;
  int64_t first;
  int b = kv8_find(c, lane, units, x, first);
  int n = kv8_len(c, b), steps = kv8_steps(c, b);
  int unit = (int)((x - first) / steps), st0 = (int)((x - first) % steps);

  while (x < x1) {
    const int st1 = (int)min((int64_t)steps, st0 + (x1 - x));
    const int h = unit / p.tiles, row0 = (unit % p.tiles) * 16 * MT;
    int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
    ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);

    // ---- queries of this unit; lim: how many cached rows each query row sees
    uint32_t qf[MT][D / 16][4];
    float mul[MT][2];
    int lim[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row0 + 16 * m + 8 * r + g;
        const int tok = row / p.a.G, hd = h * p.a.G + row % p.a.G;
        const bool ok = row < p.rows && tok < ql;
        uint32_t fr[D / 16][2];
        mul[m][r] = load_query<D>(p.a.q, b * p.a.q.sb + tok * p.a.q.st + hd * p.a.q.sh, ok, t,
                                  p.a.scale_log2, fr);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          qf[m][s][r] = fr[s][0];
          qf[m][s][2 + r] = fr[s][1];
        }
        lim[m][r] = ok ? min(n, n - ql + tok + 1) : 0;
      }

    // ---- pipeline over this warp's tiles st0 .. st1
    int64_t base[2];       // code row of the next tile's two 16-row groups, -1: none
    int64_t sbase[2];
    auto resolve = [&](int st) {
      const int pos = st * kKv8Step + warp * kSub;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        base[u] = -1;
        sbase[u] = 0;
        if (st < st1 && pos + 16 * u < n) {
          int in_page;
          const int page = kv8_page(c, b, pos + 16 * u, in_page);
          if (page >= 0) {
            base[u] = kv8_row(c, page, h, in_page);
            sbase[u] = kv8_block(c, page, h, in_page);
          } else if (lane == 0) {
            set_status(p.a.status, CSA2_DEV_BAD_PAGE);
          }
        }
      }
    };
    auto issue = [&](int st, int stage) {
      if (st < st1) {
        const int left = n - (st * kKv8Step + warp * kSub);
        uint8_t* k = ring + stage * L::kStage;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int id = lane + 32 * i, row = id / kChunks, ch = id % kChunks;
          const int64_t gb = row < 16 ? base[0] : base[1];
          const bool ok = gb >= 0 && row < left;
          const int64_t off = ok ? (gb + (row & 15)) * D + ch * 16 : 0;
          const int at = chunk_at<D>(row, ch);
          cp_async16_zfill(k + at, c.codes[0] + off, ok);
          cp_async16_zfill(k + L::kTile + at, c.codes[1] + off, ok);
        }
        float* m = reinterpret_cast<float*>(meta + stage * 32);
        if (lane < 4) {
          const int64_t sb = lane & 1 ? sbase[1] : sbase[0];
          const bool ok = (lane & 1 ? base[1] : base[0]) >= 0;
          cp_async4_zfill(m + lane, c.scales[lane >> 1] + (ok ? sb : 0), ok);
        }
        if (lane < 2) reinterpret_cast<int*>(m)[4 + lane] = (lane ? base[1] : base[0]) >= 0;
      }
      cp_async_commit();
    };

    float o[MT][kNT][4];
    float mx[MT][2], ls[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int j = 0; j < kNT; ++j) o[m][j][0] = o[m][j][1] = o[m][j][2] = o[m][j][3] = 0.0f;
      mx[m][0] = mx[m][1] = -INFINITY;
      ls[m][0] = ls[m][1] = 0.0f;
    }
    float vref = 0.0f;     // the largest V scale so far (a power of two)

    resolve(st0);
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) {
      issue(st0 + i, i);
      resolve(st0 + i + 1);
    }
    int stage = 0;
    for (int st = st0; st < st1; ++st) {
      cp_async_wait<L::kStages - 2>();
      __syncwarp();
      {
        const int nxt = st + L::kStages - 1;
        issue(nxt, stage == 0 ? L::kStages - 1 : stage - 1);
        resolve(nxt + 1);
      }
      const uint8_t* k = ring + stage * L::kStage;
      const uint8_t* v = k + L::kTile;
      const float* ms = reinterpret_cast<const float*>(meta + stage * 32);
      const float ks[2] = {ms[0], ms[1]}, vs[2] = {ms[2], ms[3]};
      const bool grp[2] = {reinterpret_cast<const int*>(ms)[4] != 0,
                           reinterpret_cast<const int*>(ms)[5] != 0};
      stage = stage + 1 == L::kStages ? 0 : stage + 1;

      // ---- S = Q K^T: four 8-row tiles of cached rows
      float s[MT][4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int m = 0; m < MT; ++m) s[m][i][0] = s[m][i][1] = s[m][i][2] = s[m][i][3] = 0.0f;
        const int row = 8 * i + key_of(g);
#pragma unroll
        for (int f = 0; f < D / 64; ++f) {
          const uint4 w = *reinterpret_cast<const uint4*>(k + chunk_at<D>(row, 4 * f + t));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t b0, b1;
            kv8_to_f16<FMT>(ww[q], b0, b1);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma16816(s[m][i], qf[m][4 * f + q], b0, b1);
          }
        }
      }

      // ---- online softmax; P in f16 times 2^15 and the V scale's share
      const float vnew = fmaxf(vref, fmaxf(vs[0], vs[1]));
      const float vdown = vnew > vref ? vref * kv8_inverse(vnew) : 1.0f;
      const float vinv = kv8_inverse(vnew);
      const float vr[2] = {vs[0] * vinv * 32768.0f, vs[1] * vinv * 32768.0f};
      vref = vnew;
      const int pos = st * kKv8Step + warp * kSub;
      uint32_t pf[MT][2][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = mx[m][r];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = pos + 8 * i + key_of(2 * t + e);
              float y = s[m][i][2 * r + e] * (mul[m][r] * ks[i >> 1]);
              if (j >= lim[m][r] || !grp[i >> 1]) y = -INFINITY;
              s[m][i][2 * r + e] = y;
              top = fmaxf(top, y);
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float use = top == -INFINITY ? 0.0f : top;
          alpha[r] = kv8_exp2(mx[m][r] - use);
          mx[m][r] = top;
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w = kv8_exp2(s[m][i][2 * r + e] - use);
              sum += w;
              s[m][i][2 * r + e] = w * vr[i >> 1];
            }
          ls[m][r] = ls[m][r] * alpha[r] + sum;
          alpha[r] *= vdown;
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              pf[m][kk][2 * u + r] =
                  pack16(s[m][2 * kk + u][2 * r], s[m][2 * kk + u][2 * r + 1], CSA2_F16);
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            o[m][j][0] *= alpha[0];
            o[m][j][1] *= alpha[0];
            o[m][j][2] *= alpha[1];
            o[m][j][3] *= alpha[1];
          }
        }
      }

      // ---- O += P V: column n of output tile j is channel (D/8) n + j
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t w[4][D / 32];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = 16 * kk + 8 * (u >> 1) + key_of(2 * t + (u & 1));
          if (D == 128) {
            const uint4 y = *reinterpret_cast<const uint4*>(v + chunk_at<D>(row, g));
            w[u][0] = y.x; w[u][1] = y.y; w[u][D / 32 - 2] = y.z; w[u][D / 32 - 1] = y.w;
          } else {
            const uint2 y =
                *reinterpret_cast<const uint2*>(v + chunk_at<D>(row, g >> 1) + 8 * (g & 1));
            w[u][0] = y.x; w[u][1] = y.y;
          }
        }
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t b0[4], b1[4];
          kv8_to_f16<FMT>(__byte_perm(w[0][q], w[1][q], 0x5140), b0[0], b0[1]);
          kv8_to_f16<FMT>(__byte_perm(w[0][q], w[1][q], 0x7362), b0[2], b0[3]);
          kv8_to_f16<FMT>(__byte_perm(w[2][q], w[3][q], 0x5140), b1[0], b1[1]);
          kv8_to_f16<FMT>(__byte_perm(w[2][q], w[3][q], 0x7362), b1[2], b1[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m) mma16816(o[m][4 * q + j], pf[m][kk], b0[j], b1[j]);
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();

    // ---- merge the warps, then write the rows or a partial result
    const bool whole = st0 == 0 && st1 == steps;
    float* part = p.a.part + (2 * (int64_t)blockIdx.x + (st0 > 0 ? 0 : 1)) * slot_floats(D);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ls[m][r] += __shfl_xor_sync(0xffffffffu, ls[m][r], 1);
        ls[m][r] += __shfl_xor_sync(0xffffffffu, ls[m][r], 2);
        if (t == 0) {
          sm[warp * 32 + 16 * m + 8 * r + g] = mx[m][r];
          sl[warp * 32 + 16 * m + 8 * r + g] = ls[m][r];
        }
      }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (warp == w) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = 16 * m + 8 * r + g;
            float top = sm[row];
#pragma unroll
            for (int u = 1; u < kWarps; ++u) top = fmaxf(top, sm[u * 32 + row]);
            // a sum of 0: no row was visible; of NaN: the query holds one
            const float f =
                ls[m][r] == 0.0f ? 0.0f : kv8_exp2(mx[m][r] - top) * (vref * 0x1p-15f);
            float* to = red + (8 * r + g) * (D + 4);
#pragma unroll
            for (int j = 0; j < kNT; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int ch = kNT * (2 * t + e) + j;
                const float y = o[m][j][2 * r + e] * f;
                to[ch] = w == 0 ? y : to[ch] + y;
              }
          }
        }
        __syncthreads();
      }
      // 8 threads per row, D / 8 channels each
      const int row = 16 * m + (tid >> 3), ch0 = (tid & 7) * (D / 8);
      float top = sm[row];
#pragma unroll
      for (int u = 1; u < kWarps; ++u) top = fmaxf(top, sm[u * 32 + row]);
      float l = 0.0f;
#pragma unroll
      for (int u = 0; u < kWarps; ++u)
        l += sl[u * 32 + row] == 0.0f ? 0.0f : sl[u * 32 + row] * kv8_exp2(sm[u * 32 + row] - top);
      const float* from = red + (tid >> 3) * (D + 4) + ch0;
      if (whole) {
        const int gr = row0 + row, tok = gr / p.a.G, hd = h * p.a.G + gr % p.a.G;
        if (gr < p.rows && tok < ql) {
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.a.out.data)) +
                          b * p.a.out.sb + tok * p.a.out.st + hd * p.a.out.sh + ch0;
#pragma unroll
          for (int i = 0; i < D / 8; i += 8) {
            uint4 y;
            y.x = pack16(from[i] * inv, from[i + 1] * inv, p.a.out.type);
            y.y = pack16(from[i + 2] * inv, from[i + 3] * inv, p.a.out.type);
            y.z = pack16(from[i + 4] * inv, from[i + 5] * inv, p.a.out.type);
            y.w = pack16(from[i + 6] * inv, from[i + 7] * inv, p.a.out.type);
            *reinterpret_cast<uint4*>(out + i) = y;
          }
          if (p.a.lse && ch0 == 0)
            p.a.lse[((int64_t)b * p.a.T + tok) * p.a.H + hd] =
                l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
        }
      } else {
        float* po = part + row * D + ch0;
#pragma unroll
        for (int i = 0; i < D / 8; i += 4)
          *reinterpret_cast<float4*>(po + i) =
              make_float4(from[i], from[i + 1], from[i + 2], from[i + 3]);
        if (ch0 == 0) {
          part[kKv8SlotRows * D + row] = top;
          part[kKv8SlotRows * (D + 1) + row] = l;
        }
      }
      __syncthreads();
    }

    // ---- next unit
    x += st1 - st0;
    st0 = 0;
    if (st1 == steps && ++unit == units && x < x1) {
      unit = 0;
      ++b;
      n = kv8_len(c, b);
      steps = kv8_steps(c, b);
    }
  }
}

// Joins the partial results of the units that several CTAs shared: one CTA of
// D threads per query row of a unit.  The order is that of the cached rows.
template <int D>
__global__ void __launch_bounds__(D) kv8_combine_kernel(DecodeParams p, int tile_rows) {
  griddep_wait();
  griddep_launch_dependents();
  const Kv8& c = p.a.c;
  const int lane = threadIdx.x & 31;
  const int units = c.heads * p.tiles;
  const int b = blockIdx.x / units, unit = blockIdx.x % units, row = blockIdx.y;
  const int h = unit / p.tiles, gr = (unit % p.tiles) * tile_rows + row;
  const int tok = gr / p.a.G, hd = h * p.a.G + gr % p.a.G;
  int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
  ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
  if (gr >= p.rows || tok >= ql) return;
  const int64_t total = kv8_total(c, lane) * units;
  const int steps = kv8_steps(c, b);
  const int64_t x0 = kv8_before(c, lane, b) * units + (int64_t)unit * steps, x1 = x0 + steps;
  const int ctas = kv8_sharers(total, p.ctas);
  const int c0 = (int)(((x0 + 1) * ctas - 1) / total), c1 = (int)((x1 * ctas - 1) / total);
  if (c0 == c1) return;
  // the unit began in CTA c0's second slot and went on in the others' first
  __shared__ float w[kKv8Ctas], red[2][D / 32];
  const int parts = c1 - c0 + 1;
  auto slot = [&](int i) { return p.a.part + (2 * (int64_t)(c0 + i) + (i == 0)) * slot_floats(D); };
  float top = -INFINITY;
  for (int i = threadIdx.x; i < parts; i += D) {
    w[i] = slot(i)[kKv8SlotRows * D + row];
    top = fmaxf(top, w[i]);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  if (lane == 0) red[0][threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < D / 32; ++k) top = fmaxf(top, red[0][k]);
  float l = 0.0f;
  for (int i = threadIdx.x; i < parts; i += D) {
    const float pl = slot(i)[kKv8SlotRows * (D + 1) + row];
    w[i] = pl == 0.0f ? 0.0f : kv8_exp2(w[i] - top);   // NaN sums stay NaN
    l += pl == 0.0f ? 0.0f : pl * w[i];
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  if (lane == 0) red[1][threadIdx.x >> 5] = l;
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) l += red[1][k];
  float o = 0.0f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) o = fmaf(slot(i)[row * D + threadIdx.x], w[i], o);
  const float y = l == 0.0f ? 0.0f : o / l;
  uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.a.out.data)) + b * p.a.out.sb +
                  tok * p.a.out.st + hd * p.a.out.sh + threadIdx.x;
  *out = (uint16_t)(pack16(y, 0.0f, p.a.out.type) & 0xFFFFu);
  if (p.a.lse && threadIdx.x == 0)
    p.a.lse[((int64_t)b * p.a.T + tok) * p.a.H + hd] =
        l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------- mass
// mass_j = decay mass_j + sum over the query rows of 2^(c q k_j - lse).  A warp
// holds 32 cached rows' codes as f16 B fragments and walks the query rows 16 at
// a time; a cached row belongs to one warp, so nothing is added atomically and
// the order of the sum is fixed.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) kv8_mass_kernel(DecodeParams p) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const Kv8& c = p.a.c;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t total = kv8_total(c, lane) * c.heads;
  const int ctas = kv8_sharers(total, p.ctas);
  if ((int)blockIdx.x >= ctas) return;
  int64_t x = total * blockIdx.x / ctas;
  const int64_t x1 = total * (blockIdx.x + 1) / ctas;
  int64_t first;
  int b = kv8_find(c, lane, c.heads, x, first);
  int n = kv8_len(c, b), steps = kv8_steps(c, b);
  int h = (int)((x - first) / steps), st = (int)((x - first) % steps);
  for (; x < x1; ++x) {
    const int pos = st * kKv8Step + warp * kSub;
    if (pos < n) {
      int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
      ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);
      uint32_t kf[4][D / 16][2];
      int64_t grow[2];
      float ks[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        grow[u] = -1;
        ks[u] = 0.0f;
        if (pos + 16 * u < n) {
          int in_page;
          const int page = kv8_page(c, b, pos + 16 * u, in_page);
          if (page >= 0) {
            grow[u] = kv8_row(c, page, h, in_page);
            ks[u] = c.scales[0][kv8_block(c, page, h, in_page)];
          } else if (lane == 0) {
            set_status(p.a.status, CSA2_DEV_BAD_PAGE);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + g;
        const bool ok = grow[i >> 1] >= 0 && pos + r < n;
#pragma unroll
        for (int f = 0; f < D / 64; ++f) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (ok)
            w = *reinterpret_cast<const uint4*>(c.codes[0] + (grow[i >> 1] + (r & 15)) * D +
                                                (4 * f + t) * 16);
          kv8_to_f16<FMT>(w.x, kf[i][4 * f][0], kf[i][4 * f][1]);
          kv8_to_f16<FMT>(w.y, kf[i][4 * f + 1][0], kf[i][4 * f + 1][1]);
          kv8_to_f16<FMT>(w.z, kf[i][4 * f + 2][0], kf[i][4 * f + 2][1]);
          kv8_to_f16<FMT>(w.w, kf[i][4 * f + 3][0], kf[i][4 * f + 3][1]);
        }
      }
      float sum[4][2] = {};
      const int rows = ql * p.a.G;
      // the first query token that sees row `pos`
      const int tok0 = max(0, pos - (n - ql));
      for (int r0 = tok0 * p.a.G / 16 * 16; r0 < rows; r0 += 16) {
        uint32_t qf[D / 16][4];
        float mul[2], lse2[2];
        int lim[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = r0 + 8 * r + g;
          const int tok = row / p.a.G, hd = h * p.a.G + row % p.a.G;
          const bool ok = row < rows;
          uint32_t fr[D / 16][2];
          mul[r] = load_query<D>(p.a.q, b * p.a.q.sb + tok * p.a.q.st + hd * p.a.q.sh, ok, t,
                                 p.a.scale_log2, fr);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            qf[s][r] = fr[s][0];
            qf[s][2 + r] = fr[s][1];
          }
          lim[r] = 0;
          lse2[r] = 0.0f;
          if (ok) {
            const float y = p.a.lse[((int64_t)b * p.a.T + tok) * p.a.H + hd];
            if (y != -INFINITY) {
              lse2[r] = y * 1.4426950408889634f;
              lim[r] = min(n, n - ql + tok + 1);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float s[4] = {};
#pragma unroll
          for (int q = 0; q < D / 16; ++q) mma16816(s, qf[q], kf[i][q][0], kf[i][q][1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = pos + 8 * i + 2 * t + e;
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (j < lim[r])
                sum[i][e] += kv8_exp2(s[2 * r + e] * (mul[r] * ks[i >> 1]) - lse2[r]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = sum[i][e];
          y += __shfl_xor_sync(0xffffffffu, y, 4);
          y += __shfl_xor_sync(0xffffffffu, y, 8);
          y += __shfl_xor_sync(0xffffffffu, y, 16);
          const int r = 8 * i + 2 * t + e;
          if (g == 0 && grow[i >> 1] >= 0 && pos + r < n) {
            float* m = c.mass + grow[i >> 1] + (r & 15);
            *m = p.a.decay == 0.0f ? y : *m * p.a.decay + y;
          }
        }
    }
    if (++st == steps) {
      st = 0;
      if (++h == c.heads && x + 1 < x1) {
        h = 0;
        ++b;
        n = kv8_len(c, b);
        steps = kv8_steps(c, b);
      }
    }
  }
}

template <int D, int MT, int FMT>
cudaError_t decode_as(const DecodeParams& p, cudaStream_t s) {
  auto kern = kv8_decode_kernel<D, MT, FMT>;
  static std::atomic<uint64_t> seen;
  cudaError_t e = kv8_prepare(kern, DecodeSmem<D>::kBytes, seen);
  if (e != cudaSuccess) return e;
  e = kv8_launch(kern, dim3(p.ctas), kThreads, DecodeSmem<D>::kBytes, s, p);
  if (e != cudaSuccess) return e;
  return kv8_launch(kv8_combine_kernel<D>, dim3(p.a.c.batch * p.a.c.heads * p.tiles, 16 * MT), D, 0, s, p,
                16 * MT);
}
template <int D, int FMT>
cudaError_t decode_of(DecodeParams p, cudaStream_t s) {
  const int mt = p.rows <= 16 ? 1 : 2;
  p.tiles = (p.rows + 16 * mt - 1) / (16 * mt);
  return mt == 1 ? decode_as<D, 1, FMT>(p, s) : decode_as<D, 2, FMT>(p, s);
}
template <int D, int FMT>
cudaError_t mass_as(const DecodeParams& p, cudaStream_t s) {
  return kv8_launch(kv8_mass_kernel<D, FMT>, dim3(p.ctas), kThreads, 0, s, p);
}

}  // namespace

size_t kv8_part_bytes(int D) { return 2 * (size_t)kKv8Ctas * slot_floats(D) * 4; }

cudaError_t launch_kv8_attn(const Kv8Attn& a, int num_sms, cudaStream_t s) {
  DecodeParams p{a, a.T * a.G, 1, 2 * num_sms < kKv8Ctas ? 2 * num_sms : kKv8Ctas};
  if (a.c.format == CSA2_KV8_E4M3)
    return a.D == 64 ? decode_of<64, CSA2_KV8_E4M3>(p, s) : decode_of<128, CSA2_KV8_E4M3>(p, s);
  return a.D == 64 ? decode_of<64, CSA2_KV8_INT8>(p, s) : decode_of<128, CSA2_KV8_INT8>(p, s);
}

cudaError_t launch_kv8_mass(const Kv8Attn& a, int num_sms, cudaStream_t s) {
  DecodeParams p{a, a.T * a.G, 1, 3 * num_sms < kKv8Ctas ? 3 * num_sms : kKv8Ctas};
  if (a.c.format == CSA2_KV8_E4M3)
    return a.D == 64 ? mass_as<64, CSA2_KV8_E4M3>(p, s) : mass_as<128, CSA2_KV8_E4M3>(p, s);
  return a.D == 64 ? mass_as<64, CSA2_KV8_INT8>(p, s) : mass_as<128, CSA2_KV8_INT8>(p, s);
}

}  // namespace csa2
