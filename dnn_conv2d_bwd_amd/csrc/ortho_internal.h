// ortho_internal.h -- plan, kernel arguments and launchers of the orthogonalised updates.
#pragma once
#include <stdint.h>

#include <vector>

#include "../../include/cbd.h"

namespace cbd {

// Split matrices: a value v is held as two halves, hi = half(v 2^e) and lo =
// half((v 2^e - hi) lo_up), with one exponent e for the matrix and lo_up 2^11 or 1.
// Rows are runs of 64 halves: hi of 32 neighbouring elements, then their lo.
//
// X is the matrix with its smaller side as rows (S of them, L columns); it is
// kept in both directions, since each product contracts along rows of both its
// operands.

// What a product C = P Q^T is for.
enum OrthoStage {
  ORTHO_SQUARE = 0,  // A = X X^T
  ORTHO_POLY = 1,    // B = a I + b A + c A A
  ORTHO_STEP = 2,    // X = B X, in both directions
  ORTHO_LAST = 3,    // the same, to the output
  ORTHO_SLICE = 4    // sums of slices of A's contracted side, for launch_ortho_join
};

struct OrthoArgs {
  const uint16_t *p, *q;     // operands: rows of ldp / ldq halves
  int64_t p_mat, q_mat;      // halves between matrices
  int32_t ldp, ldq;
  int32_t runs;              // of 32 elements along the contracted side
  int32_t tiles_m, tiles_n;  // (symmetric: n >= m of them)
  int32_t rows, cols;        // of C; past them zeros are stored
  uint16_t *c, *ct;          // C and C^T (symmetric: the same matrix)
  int64_t c_mat, ct_mat;
  int32_t ldc, ldct;
  float mul;                 // C is the products' sum times this
  float lo_up, lo_down;      // what lo is multiplied by, and 1 / that
  float p_mul, diag;         // ORTHO_POLY: and P times p_mul, and diag on the diagonal
  void* out;                 // ORTHO_LAST
  float scale;               // and the result is C times this
  int64_t out_row, out_mat;
  int32_t out_dtype, flip;   // flip: the output is C^T
  float* sums;               // ORTHO_SLICE: [matrix][tile][slice] tiles of 64 columns of 64
  int32_t slices, slice;     // how many, and runs of each but the last
};

struct OrthoSplit {
  const void* in;
  int64_t in_row, in_mat;
  int32_t rows, cols, dtype;
  double* partial;           // [matrices][kOrthoParts] sums of squares
  double eps, up;            // up = 2^e
  float lo_up;
  uint16_t *x, *xt;          // rows x cols in the input's direction, and the other
  int64_t x_mat, xt_mat;
  int32_t ldx, ldxt;
};

constexpr int kOrthoParts = 256;

// The first `count` matrices (of those left) in tiles of `tile`; count 0: none.
struct OrthoShare {
  int tile;
  int64_t count;
};

int launch_ortho_norm(const OrthoSplit& a, int64_t matrices, void* stream);
int launch_ortho_split(const OrthoSplit& a, int64_t matrices, void* stream);
// A from the sums of its slices, which are added in their order.
int launch_ortho_join(const OrthoArgs& a, int64_t matrices, void* stream);
int launch_ortho_product(const OrthoArgs& a, int stage, int tile, int64_t matrices, void* stream);

}  // namespace cbd

struct cbd_ortho_plan_s {
  cbd_ortho_problem prob;
  std::vector<double> coefficients;   // steps x 3
  int64_t s, l, sp, lp;               // sides, and their padded lengths
  cbd::OrthoShare sym[2], step[2];    // how A and B, and X, are computed
  int64_t slices, slice;              // of A's sums, in runs; slices is 1 where they are not split
  float lo_up;                        // of the split values
  // Exponents of X before each step, of A and of B.
  std::vector<int> ex, ea, eb;
};
