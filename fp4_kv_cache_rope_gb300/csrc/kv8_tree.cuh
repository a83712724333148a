// Trees of drafted tokens: parent[i] is the token that token i follows, an earlier
// one, or negative for a root.  What is no earlier token counts as a root.
#pragma once

#include "kv8.cuh"

namespace csa2 {

// How many tokens token `tok` follows.  Walks towards the root, whose tokens come
// ever earlier, so it ends.
__device__ __forceinline__ int kv8_depth(const int32_t* parent, int tok, bool& bad) {
  int depth = 0;
  for (int up = parent[tok]; up >= 0; up = parent[tok]) {
    if (up >= tok) {
      bad = true;
      break;
    }
    tok = up;
    ++depth;
  }
  return depth;
}

}  // namespace csa2
