// Which sequence of a pack a workgroup's slot belongs to.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdn {

// The last n in [0, n_seqs) with key(cu[n], n) <= slot, where keys rise and
// key(cu[0], 0) <= slot: which sequence a workgroup's slot belongs to.  A wave
// looks at 64 places at a time, so a pack of up to 64 sequences takes one trip
// to memory and one of 4096 two, where a binary search takes six and twelve,
// one after another.  Every lane of the wave takes part; the result is uniform.
template <typename F>
__device__ __forceinline__ int find_sequence(const int32_t* cu, int n_seqs, int64_t slot, F&& key) {
  int lo = 0, len = n_seqs;
  while (len > 1) {
    const int stride = (len + 63) / 64, n = lo + (int)(threadIdx.x & 63) * stride;
    const bool at_most = n < lo + len && key((int64_t)cu[n], n) <= slot;
    const int skip = (max((int)__popcll(__ballot(at_most)), 1) - 1) * stride;
    lo = __builtin_amdgcn_readfirstlane(lo + skip);
    len = min(stride, __builtin_amdgcn_readfirstlane(len - skip));
  }
  return lo;
}

}  // namespace gdn
