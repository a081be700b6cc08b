// How many pairs of SMs share the reduction of a tile of the ragged products: the launcher's choice
// of a tile's width and the kernel take the same answer from here.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__
#else
#define MOE_HOST_DEVICE
#endif

namespace moe {

// Pairs that share a tile's reduction of nk steps, `most` at most. A step takes some 600 clocks, a
// part about 12 a column to join, one after the other: sqrt(nk tile / 50) steps make the least of
// both. Joining at all costs the time of some 16 steps. (us, shared and not, 256 rows to 512 features: 16
// steps 10.6 and 8.8, 22 11.2 and 10.5, 24 11.2 and 11.1, 32 11.7 and 13.4, 49 12.5 and 18.4, 128 15.7 and
// 41.5. nk tile passes 31 bits from 2^29 rows on.)
MOE_HOST_DEVICE inline int shares(int most, int nk, int tile) {
  if (nk < 24) return 1;
  const int least = (int)sqrtf((float)nk * tile * 0.02f), n = nk / (least < 2 ? 2 : least);
  return n < 1 ? 1 : n < most ? n : most;
}

}  // namespace moe
