// expert_internal.h -- kernel arguments and launchers of the expert layer.
#pragma once
#include <stdint.h>

#include "../../include/cbd.h"

struct cbd_expert_plan_s {
  cbd_expert_problem prob;
  cbd_expert_options opt;
};

namespace cbd {

// The three operators as one product.  "m" is the contiguous side of the
// output (MFMA rows), "n" its row side, "k" the contracted side.
//   EXPERT_AK: out[t][m] = sum_k A_e[m][k] B[t][k]   A k-contiguous
//   EXPERT_AM: out[t][m] = sum_k A_e[k][m] B[t][k]   A m-contiguous
//   EXPERT_DW: out_e[n][m] = sum over rows t of e of A[t][m] B[t][n]
// Forward on [E][K][C] and bwd_data on [E][C][K] are EXPERT_AK, the other two
// EXPERT_AM.
enum ExpertForm { EXPERT_AK = 0, EXPERT_AM = 1, EXPERT_DW = 2 };

// Kernel argument, passed by value.
struct ExpertArgs {
  const void* a;     // W (AK, AM) or the rows of the contiguous side (DW)
  const void* b;     // rows
  void* out;
  const void* ends;
  int64_t a_expert;  // elements between experts of W (AK, AM)
  int64_t o_expert;  // elements between experts of dW (DW)
  int64_t lda, ldb, ldo;  // elements between rows
  int32_t T, E;
  int32_t M, N, K;   // N: DW only; K: AK and AM only
  int32_t ends64;    // ends holds 64-bit integers
  int32_t accumulate;
  int32_t whole_out;  // rows of out are 16-byte chunks on 16-byte boundaries
  int32_t tiles_m, tiles_n;
};

// What a launch looks like; chosen by expert_api.cpp, run by the kernels' files.
struct ExpertLaunch {
  int32_t kernel;  // cbd_expert_kernel
  int32_t form;    // ExpertForm
  int32_t dtype, out_dtype;
  int32_t bm, bn;  // tile
  int32_t threads;
  int32_t dma;     // operands go straight to LDS
  int64_t grid;
};

int launch_expert_generic(const ExpertArgs& a, const ExpertLaunch& l, void* stream);
int launch_expert_stream(const ExpertArgs& a, const ExpertLaunch& l, void* stream);
int launch_expert_mfma(const ExpertArgs& a, const ExpertLaunch& l, void* stream);

}  // namespace cbd
