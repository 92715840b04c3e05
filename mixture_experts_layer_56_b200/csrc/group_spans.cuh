// The row spans of ragged groups, from offsets that may hold anything.
#pragma once

#include <stdint.h>

namespace moe {

// span[0 .. groups] (shared memory) = the offsets held to [0, rows] and to the
// largest one before them, so that the groups [span[g], span[g + 1]) are
// disjoint and inside the tensors whatever the offsets are.  Every thread of
// the block calls it; it ends with a barrier.
__device__ __forceinline__ void group_spans(const int32_t* offsets, int groups, int rows,
                                            int32_t* span, int tid, int threads) {
  for (int g = tid; g <= groups; g += threads) span[g] = min(max(offsets[g], 0), rows);
  __syncthreads();
  if (tid < 32) {
    // running maximum, a run of groups per lane
    const int per = (groups + 32) / 32;
    const int beg = min(tid * per, groups + 1), end = min(beg + per, groups + 1);
    int most = 0;
    for (int i = beg; i < end; ++i) most = max(most, span[i]);
    int before = most;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (tid >= o) before = max(before, v);
    }
    before = __shfl_up_sync(0xffffffffu, before, 1);
    if (tid == 0) before = 0;
    for (int i = beg; i < end; ++i) {
      before = max(before, span[i]);
      span[i] = before;
    }
  }
  __syncthreads();
}

}  // namespace moe
