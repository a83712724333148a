// C-ABI entry points of the 8-bit K/V cache: host-side validation and launches.
// Every entry point returns a csa2_status and never throws.
#include <math.h>

#include <atomic>

#include "kv8.cuh"

using namespace csa2;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool kv8_ok(const csa2_kv8_cache* c) {
  if (!c) return false;
  if (c->batch <= 0 || c->batch > 65535 || c->kv_heads < 1 || c->kv_heads > 1024) return false;
  if (c->dim != 64 && c->dim != 128) return false;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return false;
  if (c->max_len <= 0 || c->max_len > CSA2_MAX_LEN || c->page_size < 0) return false;
  if (c->format != CSA2_KV8_E4M3 && c->format != CSA2_KV8_INT8) return false;
  if (c->page_size > 0) {
    if (c->page_size % c->block != 0 || c->page_size > CSA2_MAX_LEN) return false;
    if (!c->page_table || !aligned(c->page_table, 4) || c->max_pages_per_seq <= 0 ||
        c->num_pages <= 0)
      return false;
    if ((int64_t)c->max_pages_per_seq * c->page_size < c->max_len) return false;
  } else if (c->max_len % c->block != 0) {
    return false;
  }
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !c->seq_len) return false;
  return aligned(c->k_codes, 16) && aligned(c->v_codes, 16) && aligned(c->k_scales, 4) &&
         aligned(c->v_scales, 4) && aligned(c->mass, 4) && aligned(c->seq_len, 4);
}

Kv8 kv8_of(const csa2_kv8_cache& c) {
  Kv8 k{};
  k.codes[0] = c.k_codes;
  k.codes[1] = c.v_codes;
  k.scales[0] = c.k_scales;
  k.scales[1] = c.v_scales;
  k.mass = c.mass;
  k.page_table = c.page_table;
  k.seq_len = c.seq_len;
  k.batch = c.batch;
  k.heads = c.kv_heads;
  k.block_shift = c.block == 16 ? 4 : c.block == 32 ? 5 : c.block == 64 ? 6 : 7;
  k.paged = c.page_size > 0;
  k.page_rows = k.paged ? c.page_size : c.max_len;
  k.max_pages = k.paged ? c.max_pages_per_seq : 1;
  k.max_len = c.max_len;
  k.num_pages = k.paged ? c.num_pages : c.batch;
  k.format = c.format;
  k.page_shift = -1;
  if (k.paged && (c.page_size & (c.page_size - 1)) == 0)
    for (k.page_shift = 0; (1 << k.page_shift) < c.page_size; ++k.page_shift) {
    }
  return k;
}

bool rows_ok(const csa2_rows* r, bool wide) {
  if (!r || !r->data || !aligned(r->data, 16)) return false;
  if (r->type != CSA2_BF16 && r->type != CSA2_F16 && !(wide && r->type == CSA2_F32)) return false;
  const int64_t es = r->type == CSA2_F32 ? 4 : 2;
  return r->stride_b * es % 16 == 0 && r->stride_t * es % 16 == 0 && r->stride_h * es % 16 == 0;
}
// Whether no two rows of [B, T, H, D] overlap, by nested strides: each at least
// what the dimensions with smaller ones extend over.
bool rows_apart(const csa2_rows& r, int64_t B, int64_t T, int64_t H, int64_t D) {
  const int64_t n[3] = {B, T, H}, stride[3] = {r.stride_b, r.stride_t, r.stride_h};
  uint64_t extent = (uint64_t)D;
  bool done[3] = {B <= 1, T <= 1, H <= 1};
  auto size = [&](int i) { return stride[i] < 0 ? 0 - (uint64_t)stride[i] : (uint64_t)stride[i]; };
  for (;;) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!done[i] && (at < 0 || size(i) < size(at))) at = i;
    if (at < 0) return true;
    const uint64_t st = size(at);
    if (st < extent || st > ((uint64_t)1 << 62) / (uint64_t)n[at]) return false;
    extent += st * (uint64_t)(n[at] - 1);
    done[at] = true;
  }
}
Kv8Rows rows_of(const csa2_rows& r) {
  return Kv8Rows{r.data, r.stride_b, r.stride_t, r.stride_h, r.type};
}

// SMs of the current device, looked up once per device.
int sms() {
  static std::atomic<int> known[kKv8Devices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  if (dev >= 0 && dev < kKv8Devices && (n = known[dev].load(std::memory_order_relaxed)) > 0)
    return n;
  if (dev < 0 ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;
  }
  if (dev < kKv8Devices) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

csa2_status done(cudaError_t e) {
  if (e == cudaSuccess) return CSA2_OK;
  cudaGetLastError();   // reported here; not left for the caller's next CUDA call
  return CSA2_ERR_CUDA;
}

bool overlap(const int32_t* a, const int32_t* b, int64_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && x < y + 4 * n && y < x + 4 * n;
}

// Whether two caches whose places the host knows (at least one is contiguous)
// have storage in common.  Two paged ones may lie in one pool of pages.
bool shares_storage(const csa2_kv8_cache& a, const csa2_kv8_cache& b) {
  if (a.page_size > 0 && b.page_size > 0) return false;
  struct Range {
    uintptr_t at, end;
  };
  auto ranges = [](const csa2_kv8_cache& c, Range (&r)[5]) {
    const uintptr_t rows = (uintptr_t)(c.page_size > 0 ? c.num_pages : c.batch) * c.kv_heads *
                           (c.page_size > 0 ? c.page_size : c.max_len);
    const void* p[5] = {c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.mass};
    const uintptr_t bytes[5] = {rows * c.dim, rows * c.dim, rows / c.block * 4, rows / c.block * 4,
                                c.mass ? rows * 4 : 0};
    for (int i = 0; i < 5; ++i) {
      r[i].at = reinterpret_cast<uintptr_t>(p[i]);
      r[i].end = r[i].at + bytes[i];
    }
  };
  Range x[5], y[5];
  ranges(a, x);
  ranges(b, y);
  for (const Range& i : x)
    for (const Range& j : y)
      if (i.at < j.end && j.at < i.end) return true;
  return false;
}

struct Kv8Ws {
  size_t status, old_len, part, total;
};
Kv8Ws kv8_ws(const csa2_kv8_cache* c) {
  Kv8Ws w{};
  w.old_len = 256;
  w.part = align256(w.old_len + 4 * (size_t)c->batch);
  const size_t few = kv8_part_bytes(c->dim), many = kv8_prefill_part_bytes(c->dim);
  w.total = align256(w.part + (few > many ? few : many));
  return w;
}

bool heads_ok(const csa2_kv8_cache* c, int32_t T, int32_t H) {
  return H > 0 && H % c->kv_heads == 0 && H <= 65536 && T >= 0 && T <= CSA2_MAX_LEN &&
         (int64_t)c->batch * H * (T + 1) < (int64_t)1 << 31;
}

// The kernels' factor is the scale times log2(e), in fp32: beyond that range, and
// where it would lose bits, there is none.
bool scale_ok(float scale) {
  return scale <= 0.0f || (scale >= 0x1p-100f && scale <= 0x1p100f);
}

Kv8Attn attn_of(const csa2_kv8_cache* c, const csa2_rows* q, int32_t H, int32_t T,
                const int32_t* q_len, float scale, void* ws) {
  Kv8Attn a{};
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.c = kv8_of(*c);
  if (q) a.q = rows_of(*q);
  a.q_len = q_len;
  a.T = T;
  a.H = H;
  a.G = H / c->kv_heads;
  a.D = c->dim;
  const double to2 = (scale > 0.0f ? (double)scale : 1.0 / sqrt((double)c->dim)) * 1.4426950408889634;
  a.scale_log2 = (float)to2;
  a.scale_low = (float)(to2 - (double)a.scale_log2);
  a.part = reinterpret_cast<float*>(w + kv8_ws(c).part);
  a.status = reinterpret_cast<uint32_t*>(w);
  return a;
}

}  // namespace

extern "C" {

size_t csa2_kv8_workspace_size(const csa2_kv8_cache* cache, int32_t T, int32_t H) {
  if (!kv8_ok(cache) || !heads_ok(cache, T, H)) return 0;
  return kv8_ws(cache).total;
}

csa2_status csa2_kv8_append(const csa2_kv8_cache* cache, const csa2_rows* k, const csa2_rows* v,
                            int32_t T, const int32_t* new_len, const int32_t* start, void* ws,
                            void* stream) {
  if (!kv8_ok(cache) || !ws || !aligned(ws, 256) || T < 0 || T > CSA2_MAX_LEN)
    return CSA2_ERR_INVALID;
  if (!aligned(new_len, 4) || !aligned(start, 4)) return CSA2_ERR_INVALID;
  // seq_len is written while these are read
  if (overlap(new_len, cache->seq_len, cache->batch) ||
      (start != cache->seq_len && overlap(start, cache->seq_len, cache->batch)))
    return CSA2_ERR_INVALID;
  if (T == 0 && !start) return CSA2_OK;
  if (T > 0 && (!rows_ok(k, true) || !rows_ok(v, true) || k->type != v->type))
    return CSA2_ERR_INVALID;
  const csa2_rows none = {nullptr, 0, 0, 0, CSA2_BF16};
  return done(launch_kv8_append(kv8_of(*cache), cache->dim, rows_of(T ? *k : none),
                                rows_of(T ? *v : none), T, new_len, start,
                                static_cast<uint32_t*>(ws), (cudaStream_t)stream));
}

csa2_status csa2_kv8_attn(const csa2_kv8_cache* cache, const csa2_rows* q, int32_t H, int32_t T,
                          const int32_t* q_len, float softmax_scale, const csa2_rows* out,
                          float* lse, void* ws, void* stream) {
  if (!kv8_ok(cache) || !ws || !aligned(ws, 256) || !heads_ok(cache, T, H) || !scale_ok(softmax_scale))
    return CSA2_ERR_INVALID;
  if (!aligned(q_len, 4) || !aligned(lse, 4)) return CSA2_ERR_INVALID;
  if (T == 0) return CSA2_OK;
  if (!rows_ok(q, false) || !rows_ok(out, false) || q->type != out->type ||
      !rows_apart(*out, cache->batch, T, H, cache->dim))
    return CSA2_ERR_INVALID;
  Kv8Attn a = attn_of(cache, q, H, T, q_len, softmax_scale, ws);
  a.out = rows_of(*out);
  a.lse = lse;
  // Up to 64 query rows per (sequence, K/V head) go to the kernel that is bound by
  // the cache's bytes, more to the tensor cores' (16 sequences of 9000 rows, 4 heads,
  // D 128: 62 us against 80 us for 48 rows, 78 against 80 for 64, 92 against 82 for 80).
  return done(a.T * a.G <= 64 ? launch_kv8_attn(a, sms(), (cudaStream_t)stream)
                              : launch_kv8_prefill(a, sms(), (cudaStream_t)stream));
}

csa2_status csa2_kv8_mass(const csa2_kv8_cache* cache, const csa2_rows* q, int32_t H, int32_t T,
                          const int32_t* q_len, const float* lse, float softmax_scale, float decay,
                          void* ws, void* stream) {
  if (!kv8_ok(cache) || !cache->mass || !ws || !aligned(ws, 256) || !heads_ok(cache, T, H) ||
      !scale_ok(softmax_scale) || !(decay >= 0.0f && decay <= 1.0f))
    return CSA2_ERR_INVALID;
  if (!aligned(q_len, 4) || !aligned(lse, 4)) return CSA2_ERR_INVALID;
  if (T > 0 && (!rows_ok(q, false) || !lse)) return CSA2_ERR_INVALID;
  Kv8Attn a = attn_of(cache, T ? q : nullptr, H, T, q_len, softmax_scale, ws);
  a.lse = const_cast<float*>(lse);
  a.decay = decay;
  // Up to 32 query rows per (sequence, K/V head) stay in a warp's registers: 16
  // sequences of 9000 rows, 4 heads, D 128 take 34 us with 32 rows, the tensor
  // cores' kernel 97 us with 32 and 99 us with 64.  Up to 64 in two launches is
  // faster too (63 us with 64 rows), unless the cache is so small that the
  // launches are what takes the time (2 sequences of 2000: 24 us against 13 us).
  const int64_t tiles = (int64_t)cache->batch * cache->kv_heads * ((cache->max_len + 127) / 128);
  const int rows = T * a.G <= 32 || tiles <= 4 * (int64_t)sms() ? 32 : 64;
  return done(T * a.G <= rows ? launch_kv8_mass_few(a, sms(), (cudaStream_t)stream)
                              : launch_kv8_mass_many(a, sms(), (cudaStream_t)stream));
}

csa2_status csa2_kv8_evict(const csa2_kv8_cache* cache, const csa2_kv8_cache* dst, int32_t keep,
                           int32_t sink, int32_t recent, int32_t* kept, void* ws, void* stream) {
  if (!kv8_ok(cache) || !cache->mass || !kept || !aligned(kept, 4) || !ws || !aligned(ws, 256))
    return CSA2_ERR_INVALID;
  if (keep < 1 || sink < 0 || recent < 0 || sink > keep || recent > keep - sink)
    return CSA2_ERR_INVALID;
  const csa2_kv8_cache* d = dst ? dst : cache;
  if (dst && (!kv8_ok(dst) || dst->batch != cache->batch || dst->kv_heads != cache->kv_heads ||
              dst->dim != cache->dim || dst->block != cache->block ||
              dst->format != cache->format ||
              overlap(dst->seq_len, cache->seq_len, cache->batch) || shares_storage(*cache, *dst)))
    return CSA2_ERR_INVALID;
  if (keep > d->max_len) return CSA2_ERR_INVALID;
  uint8_t* w = static_cast<uint8_t*>(ws);
  return done(launch_kv8_evict(kv8_of(*cache), kv8_of(*d), dst == nullptr, cache->dim, keep, sink,
                               recent, kept, reinterpret_cast<int32_t*>(w + kv8_ws(cache).old_len),
                               reinterpret_cast<uint32_t*>(w), sms(), (cudaStream_t)stream));
}

}  // extern "C"
