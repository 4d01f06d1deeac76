// Which tiles of a list a persistent workgroup takes, and the wait for its loads, shared by the grouped GEMMs on
// quantised weights.
#pragma once

#include "common.h"

namespace moe {

// This workgroup's tiles out of `total`: the list is cut into eight contiguous ranges, one per XCD (workgroup b runs
// on XCD b % 8), so tiles that share weights or rows meet in one L2.
struct Tiles {
  int begin, end, step;
};
__device__ __forceinline__ Tiles my_tiles(int total) {
  const int G = gridDim.x;
  Tiles t{(int)blockIdx.x, total, G};
  if ((G & 7) == 0) {
    const int x = blockIdx.x & 7, per = (total + 7) >> 3;
    t.begin = x * per + (blockIdx.x >> 3);
    t.end = min(total, (x + 1) * per);
    t.step = G >> 3;
  }
  return t;
}

// Until at most N of this wave's loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace moe
