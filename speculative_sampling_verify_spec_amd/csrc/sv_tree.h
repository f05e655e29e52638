// Ancestor sets of token-tree nodes, for the verification, the mask and the
// attention.
#pragma once

#include "sv_internal.h"

namespace sv {

// Lane v < n: the ancestor set of node v of tree `par` (n <= 64 nodes),
// its validity (parent in [0, v)) and its depth.
__device__ inline void ancestor_sets(const int32_t* par, int n, uint64_t& set, bool& valid, int& depth) {
  const int v = threadIdx.x % kWave;
  const int pv = v < n ? par[v] : -1;
  valid = v == 0 || (v < n && pv >= 0 && pv < v);
  set = v < n ? (1ull << v) : 0ull;
  int jump = (v < n && v > 0 && valid) ? pv : -1;
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    const uint64_t up = __shfl(set, jump < 0 ? v : jump, kWave);
    const int jj = __shfl(jump, jump < 0 ? v : jump, kWave);
    if (jump >= 0) {
      set |= up;
      jump = jj;
    }
  }
  depth = __popcll(set) - 1;
}

}  // namespace sv
