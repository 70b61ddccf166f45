// What the differential-attention kernels share.  A head's D columns of q and k hold the
// two maps' d = D / 2 side by side, so all else is as in the cross attention: the packing
// of the rows that share a key head into tiles, strides, lengths and runs.
#pragma once

#include "cross_common.cuh"
#include "internal.h"

namespace nabla {
namespace diff {

constexpr int kStates = 64;  // states per tile

// 16-state MMA steps of tile t of a batch with `len` states: 4, or fewer in its last tile.
__device__ __forceinline__ int steps16(int len, int t) {
  const int left = len - t * kStates;
  return left >= kStates ? 4 : (left + 15) >> 4;
}

// Rows [rows, end) of a tile (128 bytes a row and box) as zeros; a whole warp.
template <int kBoxes>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int box, int rows, int end) {
  const int n16 = (end - rows) * 8;
  for (int c = 0; c < kBoxes; ++c)
    for (int e = threadIdx.x & 31; e < n16; e += 32)
      *reinterpret_cast<uint4 *>(tile + c * box + rows * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
  tc::fence_async_smem();
  __syncwarp();
}

// 16-column step kk (of all D columns) of a K-major tile of `box` bytes a box.
__device__ __forceinline__ uint64_t k_step(int kk, int box) {
  return (uint64_t)(((kk >> 2) * box + (kk & 3) * 32) >> 4);
}

}  // namespace diff
}  // namespace nabla
