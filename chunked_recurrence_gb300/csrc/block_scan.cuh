// block_scan.cuh -- sums over a block's threads, compiled for the device by the kernels and for the host by the tests, which run
// a block's threads one after another.
#pragma once

#include <stdint.h>

namespace gdn {
namespace pages {

// Inclusive sum over the block's threads; *total gets the whole.  sh: 33 words.
__device__ __forceinline__ int block_scan(int x, int *sh, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  __syncthreads();  // sh is free
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = lane < warps ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += u;
    }
    sh[lane] = y;
  }
  __syncthreads();
  *total = sh[warps - 1];
  return x + (warp ? sh[warp - 1] : 0);
}

}  // namespace pages
}  // namespace gdn
