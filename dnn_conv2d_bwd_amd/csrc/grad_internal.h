// grad_internal.h -- kernel arguments and launchers of the gradient norm and
// clipping.
#pragma once
#include <stdint.h>

#include <vector>

#include "../../include/cbd.h"

namespace cbd {

// Tensors of one launch: pointers travel in the kernel arguments (4 KiB), so
// a call copies nothing to the device and can be captured.
constexpr int kGradBatch = 112;
constexpr int kGradChunkBytes = 1 << 16;  // one workgroup's step
// Lists up to which one workgroup does it all.  A call from Python costs what
// the host does, and a launch is 2.3 us of it: norm of 12 tensors of 480 KB
// 12.4 us a call against 15.0 with two launches.  In a graph the kernels count:
// norm of 48, 240 and 480 KB 4.3, 5.6 and 7.1 us, against 4.9 with two (of 960
// KB); clipping 48 and 120 KB 5.4 and 6.5 us against 5.5 (of 240 KB).
constexpr int kGradSmallChunks = 16;
constexpr int64_t kGradSmallNorm = 1 << 19, kGradSmallClip = 1 << 17;  // bytes
constexpr int kGradMaxGrid = 2048;        // workgroups, and partial sums, per launch: 8 per compute unit

struct GradEntry {
  const void* in;
  void* out;
  int64_t count;
  uint32_t chunk_begin;  // chunks of the batch's tensors before this one
  int32_t dtype;
};
struct GradArgs {
  GradEntry t[kGradBatch];
  double* partial;       // of the whole call
  float* norm;
  double max_norm;
  uint32_t first;        // this launch's first partial (norm pass)
  uint32_t partials;     // of the whole call
  int32_t n;             // tensors in the batch
  uint32_t chunks;
};
static_assert(sizeof(GradArgs) <= 4088, "kernel arguments");

struct GradBatch {
  int32_t begin, n;  // tensors
  uint32_t chunks, grid, first;
};

int launch_grad_partial(const GradArgs& a, uint32_t grid, void* stream);
int launch_grad_finish(const GradArgs& a, void* stream);  // norm alone
int launch_grad_small(const GradArgs& a, int clip, void* stream);  // one workgroup does it all
int launch_grad_scale(const GradArgs& a, uint32_t grid, void* stream);

}  // namespace cbd

struct cbd_grad_plan_s {
  std::vector<int64_t> counts;
  std::vector<int32_t> dtypes;
  std::vector<int32_t> index;           // non-empty tensors
  std::vector<uint32_t> chunk_begin;    // of each of those, within its batch
  std::vector<cbd::GradBatch> batches;  // ranges of index
  uint32_t partials = 0;
  int64_t bytes = 0;
};
