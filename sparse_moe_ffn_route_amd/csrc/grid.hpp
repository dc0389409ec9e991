// Grids of more workgroups than one dimension holds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// A grid dimension holds less than 2^32 threads; a launch of more runs in part, without an error.  Grids that
// grow with the tokens have 2^20 workgroups to a row and as many rows as they need, the last with some to spare.
inline dim3 wide_grid(int64_t blocks) {
  constexpr int64_t kRow = 1 << 20;
  const int64_t x = blocks < kRow ? blocks : kRow;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x));
}
__device__ __forceinline__ int wide_block() { return static_cast<int>(blockIdx.y * gridDim.x + blockIdx.x); }

}  // namespace moe
