// scan.cuh -- a prefix sum over the threads of a planning CTA.
#pragma once

#include <stdint.h>

namespace fp8pa {

namespace {

constexpr int kPlanThreads = 1024;

// Exclusive scan of one int per thread over the CTA; returns the total.
__device__ __forceinline__ int block_scan(int x, int* excl, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *excl = v - x + (warp ? s_warp[warp - 1] : 0);
  const int total = s_warp[kPlanThreads / 32 - 1];
  __syncthreads();
  return total;
}

}  // namespace

}  // namespace fp8pa
