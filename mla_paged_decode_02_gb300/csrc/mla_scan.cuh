// mla_scan.cuh — the block-wide prefix sum of the schedulers (1024 threads).
#pragma once
#include <cstdint>

namespace mla {

constexpr int kSchedThreads = 1024;

// Exclusive prefix sum over the block's threads (warp shuffles, then the 32 warp totals).
__device__ __forceinline__ int64_t block_exclusive_scan(int64_t v, int64_t* tmp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = tmp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += y;
    }
    tmp[lane] = w;                         // inclusive totals of warps 0..lane
  }
  __syncthreads();
  const int64_t before = (warp > 0 ? tmp[warp - 1] : 0) + x - v;
  *total = tmp[31];
  __syncthreads();
  return before;
}

}  // namespace mla
