// The many-row attention over the 8-bit K/V cache with changed scores, and of
// drafted tokens over the cached rows.
#include "kv8_prefill.cuh"

namespace csa2 {

cudaError_t launch_kv8_scored_many(const Kv8Attn& a, const Kv8Scores& sc, int num_sms, Kv8Left* left,
                                   cudaStream_t s) {
  if (sc.cap2 > 0.0f)
    return sc.slopes ? prefill_any<kBoth>(a, sc, num_sms, s, left)
                     : prefill_any<kCapped>(a, sc, num_sms, s, left);
  return sc.slopes ? prefill_any<kSloped>(a, sc, num_sms, s, left)
                   : prefill_any<kMasked>(a, sc, num_sms, s, left);
}

cudaError_t set_wait_limit_kv8_scored(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace csa2
