// Warp-level top-16 selection over (value, id) keys, shared by the kernels
// that scan logits.
#pragma once

#include "common.cuh"

namespace dflash {

constexpr int TOP_K = 16;

// Warp-wide sorted list in lanes 0..15 (descending).  Insert key k (uniform).
__device__ __forceinline__ void insert(uint64_t &list, uint64_t k, int lane) {
  const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
  if (lane < TOP_K) list = (list > k) ? list : ((lane == 0 || up > k) ? k : up);
}

// Offer one key per lane; inserts every key that beats the current 16th.
__device__ __forceinline__ void offer(uint64_t &list, uint64_t &thr, uint64_t key, int lane) {
  unsigned m = __ballot_sync(0xffffffffu, key > thr);
  while (m) {
    const int src = __ffs(m) - 1;
    const uint64_t k = __shfl_sync(0xffffffffu, key, src);
    insert(list, k, lane);
    thr = __shfl_sync(0xffffffffu, list, TOP_K - 1);
    m &= ~(1u << src);
    m &= __ballot_sync(0xffffffffu, key > thr);
  }
}

// The 16th largest of the 32 lanes' values (a warp-wide descending bitonic
// sort; every lane gets the result).
__device__ __forceinline__ float warp_16th_largest(float v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, j);
      const bool up = ((lane & k) == 0) == ((lane & j) == 0);   // this lane keeps the larger
      v = up ? fmaxf(v, o) : fminf(v, o);
    }
  }
  return __shfl_sync(0xffffffffu, v, TOP_K - 1);
}

}  // namespace dflash
