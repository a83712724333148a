// The few-row attention over the 8-bit K/V cache, and the weights that each cached
// row gets from few query rows.
#include "kv8_decode.cuh"

namespace csa2 {
namespace {

// ---------------------------------------------------------------------- mass
// CTAs that an SM holds, by the registers of the query rows.
constexpr int mass_ctas(int nt) { return nt == 1 ? 4 : nt == 2 ? 3 : 2; }

// mass_j = decay mass_j + sum over the query rows of 2^(c q k_j - lse), for
// 8 NT query rows from row0 on: their fragments stay in registers while a warp streams its
// cached rows, the next tile's codes loaded while this one is worked on.  A
// cached row belongs to one warp, so nothing is added atomically and the order
// of the sum is fixed.
//
// The exponent is x = s f - hi with f = (1 - eps) c log2(e) 2^e s_K as rounded and
// lse log2(e) = hi + lo; what the roundings leave goes into the factor
// 2^(eps hi - lo) of the sum (but for eps x, nothing for the weights that count).
// At logits of 20 to 30 it is 1e-6 of the weight.
template <int D, int NT, int FMT>
__global__ void __launch_bounds__(kThreads, mass_ctas(NT)) kv8_mass_kernel(DecodeParams p) {
  constexpr int kHalf = D / 64;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const Kv8& c = p.a.c;
  griddep_wait();
  griddep_launch_dependents();
  const Kv8Share first = kv8_share(c, lane, c.heads, p.ctas, blockIdx.x);
  if ((int)blockIdx.x >= first.ctas) return;
  int64_t x = first.x;
  const int64_t x1 = first.x1;
  int b = first.b, n = first.n, steps = first.steps, h = first.unit, st0 = first.step;
  while (x < x1) {
    const int st1 = (int)min((int64_t)steps, st0 + (x1 - x));
    int ql = p.a.q_len ? p.a.q_len[b] : p.a.T;
    ql = ql < 0 ? 0 : (ql > p.a.T ? p.a.T : ql);

    // one tile's codes are on their way while another is worked on, and the page
    // ids of one more
    struct Tile {
      Groups at;
      uint4 raw[2][kHalf][2];   // rows 16 i + 8 r + g, 16-byte chunk 4 f + t
      float ks[2];
    };
    Tile tile;
    int id;
    auto fetch = [&](int st) {
      id = fetch_page(c, b, st * kKv8Step + warp * kSub, st < st1 ? n : 0, lane);
    };
    auto load = [&](Tile& x, int st) {
      const int pos = st * kKv8Step + warp * kSub;
      x.at = place_groups(c, id, h, pos, p.a.status, lane);
      fetch(st + 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.ks[i] = 0.0f;
        if (x.at.row[i] >= 0) x.ks[i] = c.scales[0][x.at.blk[i]];
#pragma unroll
        for (int f = 0; f < kHalf; ++f)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            x.raw[i][f][r] = make_uint4(0, 0, 0, 0);
            if (x.at.row[i] >= 0 && pos + 16 * i + 8 * r + g < n)
              x.raw[i][f][r] = *reinterpret_cast<const uint4*>(
                  c.codes[0] + (x.at.row[i] + 8 * r + g) * D + (4 * f + t) * 16);
          }
      }
    };
    fetch(st0);
    load(tile, st0);

    uint32_t qf[NT][D / 16][2];
    float mul[NT][2], l2[NT][2], gain[NT][2];
    const float eps = p.a.scale_low / p.a.scale_log2;
    int lim[NT][2], full = 0x7FFFFFFF;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int row = p.row0 + 8 * u + g, tok = row / p.a.G, hd = h * p.a.G + row % p.a.G;
      const bool ok = row < p.rows && tok < ql;
      const float f = load_query<D>(p.a.q, b * p.a.q.sb + tok * p.a.q.st + hd * p.a.q.sh, ok, t,
                                    1.0f, qf[u]);
      const float y = ok ? p.a.lse[((int64_t)b * p.a.T + tok) * p.a.H + hd] : -INFINITY;
      const int see = ok && fabsf(y) != INFINITY ? max(0, min(n, n - ql + tok + 1)) : 0;
      // a row without weight: a constant so large that every weight is 0, and a
      // zero row, because a NaN or an infinity in it would still count
      if (see == 0) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) qf[u][i][0] = qf[u][i][1] = 0u;
      }
      const float hi = see ? y * 1.44269502f : INFINITY;
      const float g2 =
          see ? exp2f(eps * hi - (fmaf(y, 1.44269502f, -hi) + y * 1.92596299e-8f)) : 1.0f;
      if (see) full = min(full, see);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from = 4 * (2 * t + e);
        const float fe = __shfl_sync(0xffffffffu, f, from);
        mul[u][e] = p.a.scale_log2 * fe;
        l2[u][e] = __shfl_sync(0xffffffffu, hi, from);
        gain[u][e] = __shfl_sync(0xffffffffu, g2, from);
        lim[u][e] = __shfl_sync(0xffffffffu, see, from);
      }
    }
    full = __reduce_min_sync(0xffffffffu, full);

    for (int st = st0; st < st1; ++st) {
      const int pos = st * kKv8Step + warp * kSub;
      const Groups here = tile.at;
      const float kscale[2] = {tile.ks[0], tile.ks[1]};
      // The logits in two chains of products that are added at the end: what the
      // tensor cores cut off at each step adds up over fewer steps (the weights'
      // error: 1.5e-6 in one chain at logits of 20 to 30).
      float s[NT][2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float half[2][NT][4];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) half[0][u][e] = half[1][u][e] = 0.0f;
#pragma unroll
        for (int f = 0; f < kHalf; ++f) {
          const uint32_t* xa = reinterpret_cast<const uint32_t*>(&tile.raw[i][f][0]);
          const uint32_t* xb = reinterpret_cast<const uint32_t*>(&tile.raw[i][f][1]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t a[4];
            kv8_to_f16<FMT>(xa[q], a[0], a[2]);
            kv8_to_f16<FMT>(xb[q], a[1], a[3]);
#pragma unroll
            for (int u = 0; u < NT; ++u)
              mma16816(half[q & 1][u], a, qf[u][4 * f + q][0], qf[u][4 * f + q][1]);
          }
        }
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][i][e] = half[0][u][e] + half[1][u][e];
      }
      load(tile, st + 1);
      const bool some = pos + kSub > full;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 16 * i + 8 * r + g;
          float sum = 0.0f;
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float z = s[u][i][2 * r + e] * kscale[i];       // exact: a power of two
              const float w = kv8_exp2(fmaf(z, mul[u][e], -l2[u][e]));
              // (a hidden weight is left out and not taken as 0: its gain may be NaN)
              const float with = fmaf(w, gain[u][e], sum);
              sum = some && pos + row >= lim[u][e] ? sum : with;
            }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if (t == 0 && here.row[i] >= 0 && pos + row < n) {
            float* m = c.mass + here.row[i] + 8 * r + g;
            *m = p.a.decay == 0.0f ? sum : *m * p.a.decay + sum;
          }
        }
    }
    x += st1 - st0;
    st0 = 0;
    if (st1 == steps && ++h == c.heads && x < x1) {
      h = 0;
      ++b;
      n = kv8_len(c, b);
      steps = kv8_steps(c, b);
    }
  }
}

template <int D, int NT, int FMT>
cudaError_t mass_as(DecodeParams p, int num_sms, cudaStream_t s) {
  const int ctas = mass_ctas(NT) * num_sms;
  p.ctas = ctas < kKv8Ctas ? ctas : kKv8Ctas;
  return kv8_launch(kv8_mass_kernel<D, NT, FMT>, dim3(p.ctas), kThreads, 0, s, p);
}
template <int D, int FMT>
cudaError_t mass_of(const DecodeParams& p, int num_sms, cudaStream_t s) {
  const int rows = p.rows - p.row0;
  return rows <= 8    ? mass_as<D, 1, FMT>(p, num_sms, s)
         : rows <= 16 ? mass_as<D, 2, FMT>(p, num_sms, s)
                      : mass_as<D, 4, FMT>(p, num_sms, s);
}
template <int FMT>
cudaError_t mass_rows(DecodeParams p, int num_sms, cudaStream_t s) {
  do {   // 32 query rows at a time; those behind the first add to what they left
    const cudaError_t e =
        p.a.D == 64 ? mass_of<64, FMT>(p, num_sms, s) : mass_of<128, FMT>(p, num_sms, s);
    if (e != cudaSuccess) return e;
    p.row0 += 32;
    p.a.decay = 1.0f;
  } while (p.row0 < p.rows);
  return cudaSuccess;
}

}  // namespace

size_t kv8_part_bytes(int D) { return 2 * (size_t)kKv8Ctas * slot_floats(D) * 4; }

cudaError_t launch_kv8_attn(const Kv8Attn& a, int num_sms, cudaStream_t s) {
  const DecodeParams p{a, a.T * a.G, 1, 1, 0, {}};
  if (a.c.format == CSA2_KV8_E4M3)
    return a.D == 64 ? decode_of<64, CSA2_KV8_E4M3, false>(p, num_sms, s)
                     : decode_of<128, CSA2_KV8_E4M3, false>(p, num_sms, s);
  return a.D == 64 ? decode_of<64, CSA2_KV8_INT8, false>(p, num_sms, s)
                   : decode_of<128, CSA2_KV8_INT8, false>(p, num_sms, s);
}

cudaError_t launch_kv8_mass_few(const Kv8Attn& a, int num_sms, cudaStream_t s) {
  const DecodeParams p{a, a.T * a.G, 1, 1, 0, {}};
  return a.c.format == CSA2_KV8_E4M3 ? mass_rows<CSA2_KV8_E4M3>(p, num_sms, s)
                                     : mass_rows<CSA2_KV8_INT8>(p, num_sms, s);
}

}  // namespace csa2
