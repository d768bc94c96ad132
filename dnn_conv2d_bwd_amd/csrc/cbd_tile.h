// cbd_tile.h -- which tile a workgroup computes.
#pragma once

namespace cbd {
namespace dev {

// Logical tile of hardware workgroup b.  Workgroups are dealt round-robin to
// the 8 XCDs (each with its own L2); with remap on, XCD x receives the
// contiguous logical range [x*q + min(x, r), ...), so neighbouring tiles --
// which share operand panels -- meet in one L2.
__device__ inline int logical_tile(int b, int total, int remap) {
  const int q = total >> 3, r = total & 7, x = b & 7, idx = b >> 3;
  return remap ? x * q + (x < r ? x : r) + idx : b;
}

}  // namespace dev
}  // namespace cbd
