// The many-row attention over the 8-bit K/V cache.
#include "kv8_prefill.cuh"

namespace csa2 {

size_t kv8_prefill_part_bytes(int D) { return (size_t)kKv8SplitCtas * kTileRows * (D + 2) * 4; }

cudaError_t launch_kv8_prefill(const Kv8Attn& a, int num_sms, cudaStream_t s) {
  return prefill_any<kPlain>(a, Kv8Scores{}, num_sms, s, nullptr);
}

cudaError_t set_wait_limit_kv8_prefill(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace csa2
