// block_internal.h -- plan, kernel arguments and launchers of the norms around a block.
#pragma once
#include <stdint.h>

#include "../../include/cbd.h"

namespace cbd {

// How a row of c elements is dealt out: `lanes` threads of up to `chunks`
// 16-byte chunks each.  Up to 64 lanes: several rows in a workgroup of 256
// threads; otherwise a workgroup a row.
struct BlockShape {
  int32_t lanes, chunks;
};

// Joins bwd's partial sums: sums[0] = sum dn * zn, sums[1] = sum scale * dz' * yn (* gate, of rows).
struct BlockFinish {
  const float* partial;
  const void *gate, *w_post;         // vectors
  void *dw_post, *dgate, *dw_pre;    // NULL: not wanted
  int32_t n, c, dtype, dw_dtype;     // n: workgroups
};

struct BlockArgs {
  const void *r, *y, *gate, *w_post, *w_pre;  // gate: a vector, or rows (gate_rows != 0); bwd: w_pre only with dn
  const void *dz, *dn;                        // bwd; NULL: zeros
  void *z, *n;                                // forward; NULL: not written
  void *dr, *dy, *dgate;                      // bwd; dgate: of a gate of rows
  float* stats;                               // [rows][2]: 1 / rms of y and of z
  float* partial;                             // bwd: [grid][2][c] sums; NULL: none
  int64_t ldr, ldy, ldgate, ldz, ldn, lddz, lddn, lddr, lddy, lddgate;
  int64_t rows;
  int32_t c;
  int32_t gate_rows;  // the gate has rows
  float eps, scale;
  BlockFinish finish;  // bwd by one workgroup: what it does itself in the end
};

int launch_block_forward(const BlockArgs& a, BlockShape s, int dtype, int64_t grid, void* stream);
int launch_block_bwd(const BlockArgs& a, BlockShape s, int dtype, int64_t grid, void* stream);
int launch_block_finish(const BlockFinish& a, void* stream);

// 16-byte chunks of c elements, and the shape that covers them.
constexpr int kBlockMaxC = 16384;
inline BlockShape block_shape(int64_t c, int es) {
  const int64_t chunks = (c * es + 15) / 16;
  for (int lanes = 8; lanes <= 1024; lanes *= 2)
    if (chunks <= lanes) return {lanes, 1};
  return {1024, chunks <= 2048 ? 2 : 4};
}
// Backward, whether a thread holds its columns' sums in registers, or in LDS.
constexpr bool block_held(int chunks, int es) { return chunks * 16 / es <= 8; }
// Rows that one f32 sum of a column takes at most.
constexpr int kBlockJoin = 128;
inline int block_threads(BlockShape s) { return s.lanes <= 64 ? 256 : s.lanes; }

}  // namespace cbd

struct cbd_block_plan_s {
  cbd_block_problem prob;
  cbd::BlockShape shape;
  int64_t grid_fwd, grid_bwd;
};
