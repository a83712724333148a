// The few-row attention over the 8-bit K/V cache with changed scores, and of drafted
// tokens over the cached rows.
#include "kv8_decode.cuh"

namespace csa2 {

cudaError_t launch_kv8_scored_few(const Kv8Attn& a, const Kv8Scores& sc, int num_sms, Kv8Left* left,
                                  cudaStream_t s) {
  const DecodeParams p{a, a.T * a.G, 1, 1, 0, sc};
  if (left) *left = Kv8Left{0, 0, 0, 0};
  if (a.c.format == CSA2_KV8_E4M3)
    return a.D == 64 ? decode_of<64, CSA2_KV8_E4M3, true>(p, num_sms, s, left)
                     : decode_of<128, CSA2_KV8_E4M3, true>(p, num_sms, s, left);
  return a.D == 64 ? decode_of<64, CSA2_KV8_INT8, true>(p, num_sms, s, left)
                   : decode_of<128, CSA2_KV8_INT8, true>(p, num_sms, s, left);
}

}  // namespace csa2
