// Grids of the serving step's kernels. Workgroups of a launch lie in rows of kGridRow along the grid's second dimension:
// the runtime takes fewer than 2^32 threads along the first. The last row may have some to spare, which have no work.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kamera {

constexpr int64_t kGridRow = int64_t(1) << 22;
// Workgroups that a launch of `blocks` has, those to spare among them.
constexpr int64_t grid_blocks(int64_t blocks) { return blocks <= kGridRow ? blocks : (blocks + kGridRow - 1) / kGridRow * kGridRow; }
inline dim3 grid_of(int64_t blocks, unsigned z = 1) {
  return blocks <= kGridRow ? dim3((unsigned)blocks, 1, z) : dim3((unsigned)kGridRow, (unsigned)(grid_blocks(blocks) / kGridRow), z);
}
#ifdef __HIPCC__
__device__ __forceinline__ uint32_t block_number() { return blockIdx.y * (uint32_t)kGridRow + blockIdx.x; }
#endif

}  // namespace kamera
