// mamba_grid.h -- launches of more workgroups than one grid dimension takes.
//
// A dispatch counts threads in 32 bits per dimension, and a larger product of workgroups and threads wraps
// without an error: the workgroups past it never run.  wide_grid lays such a launch out in z as well; in the kernel,
// wide_index numbers the workgroups in dispatch order, and those at or past `blocks` have nothing to do.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

namespace mamba {

constexpr uint64_t kGridThreads = (uint64_t)1 << 31;  // of a grid's x (a multiple of every workgroup x 8 XCDs)

// `blocks` < 2^32 workgroups of `threads`; y as given
inline dim3 wide_grid(uint64_t blocks, uint32_t threads, uint32_t y = 1) {
  const uint64_t most = kGridThreads / threads / 8 * 8;
  return dim3((uint32_t)std::min(blocks, most), y, (uint32_t)((blocks + most - 1) / most));
}
__device__ __forceinline__ uint32_t wide_index() { return blockIdx.z * gridDim.x + blockIdx.x; }

}  // namespace mamba
