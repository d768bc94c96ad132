// grad_api.cpp -- plans, argument checks and launches of the gradient norm
// and clipping.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <memory>
#include <string>

#include "cbd_internal.h"
#include "grad_internal.h"

namespace {

cbd_status fail(cbd_status s, const char* msg) {
  cbd::set_error(msg);
  return s;
}

template <typename F>
cbd_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return CBD_ERR_NO_MEMORY;
  }
}

int esize(int dtype) { return dtype == CBD_F32 ? 4 : 2; }

cbd_status make_plan(const int64_t* counts, const int32_t* dtypes, int32_t n, cbd_grad_plan_t** out) {
  if (!out) return fail(CBD_ERR_INVALID_ARG, "NULL output");
  *out = nullptr;
  if (n < 0 || (n > 0 && (!counts || !dtypes))) return fail(CBD_ERR_INVALID_ARG, "NULL list or negative length");
  if (n > 65536) return fail(CBD_ERR_UNSUPPORTED, "more than 65536 tensors");
  for (int32_t i = 0; i < n; i++) {
    if (counts[i] < 0) return fail(CBD_ERR_INVALID_ARG, "negative element count");
    if (dtypes[i] != CBD_F32 && dtypes[i] != CBD_BF16) return fail(CBD_ERR_INVALID_ARG, "unknown dtype");
    if (counts[i] >= (int64_t(1) << 40)) return fail(CBD_ERR_UNSUPPORTED, "a tensor of 2^40 elements or more");
  }
  std::unique_ptr<cbd_grad_plan_s> p(new cbd_grad_plan_s);
  p->counts.assign(counts, counts + n);
  p->dtypes.assign(dtypes, dtypes + n);
  for (int32_t i = 0; i < n; i++) {
    if (!counts[i]) continue;
    const uint64_t chunks = ((uint64_t)counts[i] * esize(dtypes[i]) + cbd::kGradChunkBytes - 1) / cbd::kGradChunkBytes;
    if (p->batches.empty() || p->batches.back().n == cbd::kGradBatch ||
        p->batches.back().chunks + chunks > (uint64_t(1) << 30))
      p->batches.push_back({(int32_t)p->index.size(), 0, 0, 0, 0});
    cbd::GradBatch& b = p->batches.back();
    if (chunks > (uint64_t(1) << 30)) return fail(CBD_ERR_UNSUPPORTED, "a tensor is too large");
    p->index.push_back(i);
    p->bytes += counts[i] * esize(dtypes[i]);
    p->chunk_begin.push_back(b.chunks);
    b.n++;
    b.chunks += (uint32_t)chunks;
  }
  for (cbd::GradBatch& b : p->batches) {
    b.grid = std::min<uint32_t>(b.chunks, cbd::kGradMaxGrid);
    b.first = p->partials;
    p->partials += b.grid;
  }
  *out = p.release();
  cbd::set_error("");
  return CBD_OK;
}

struct Range {
  uintptr_t p;
  uint64_t bytes;
  int32_t tensor;
  bool out;
};

cbd_status run(const cbd_grad_plan_t* plan, const void* const* grads, void* const* outs, bool clip,
               double max_norm, float* norm, void* ws, uint64_t ws_bytes, void* stream) {
  if (!plan || !norm || !ws) return fail(CBD_ERR_INVALID_ARG, "NULL plan, norm or workspace");
  const int32_t n = (int32_t)plan->counts.size();
  if (n > 0 && !grads) return fail(CBD_ERR_INVALID_ARG, "NULL list of gradients");
  if (clip && !(max_norm >= 0.0)) return fail(CBD_ERR_INVALID_ARG, "max_norm must be a number >= 0");
  uint64_t need = 0;
  cbd_grad_workspace_size(plan, &need);
  if (ws_bytes < need) return fail(CBD_ERR_INVALID_ARG, "workspace smaller than cbd_grad_workspace_size");
  if ((uintptr_t)ws & 255u) return fail(CBD_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  if ((uintptr_t)norm & 3u) return fail(CBD_ERR_UNSUPPORTED, "norm must be 4-byte aligned");
  for (int32_t i : plan->index) {
    const uintptr_t mask = (uintptr_t)esize(plan->dtypes[i]) - 1;
    if (!grads[i] || (outs && !outs[i])) return fail(CBD_ERR_INVALID_ARG, "NULL tensor pointer");
    if ((uintptr_t)grads[i] & mask || (outs && (uintptr_t)outs[i] & mask))
      return fail(CBD_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
  }
  // What is written (outputs, norm, workspace) may overlap nothing but, for an
  // output, its own gradient exactly.  Sorted by address, with the furthest
  // end of the ranges read and of those written so far.
  {
    std::vector<Range> r;
    r.reserve(2 * plan->index.size() + 2);
    r.push_back({(uintptr_t)norm, 4, -1, true});
    r.push_back({(uintptr_t)ws, need, -2, true});
    for (int32_t i : plan->index) {
      const uint64_t bytes = (uint64_t)plan->counts[i] * esize(plan->dtypes[i]);
      const void* o = !clip ? nullptr : outs ? outs[i] : grads[i];
      if (o != grads[i]) r.push_back({(uintptr_t)grads[i], bytes, i, false});
      if (o) r.push_back({(uintptr_t)o, bytes, i, true});
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.p < b.p; });
    uintptr_t read_end = 0, write_end = 0;
    for (const Range& x : r) {
      if (x.p < write_end || (x.out && x.p < read_end))
        return fail(CBD_ERR_INVALID_ARG, "an output, norm or the workspace overlaps another tensor");
      uintptr_t& end = x.out ? write_end : read_end;
      end = std::max<uintptr_t>(end, x.p + x.bytes);
    }
  }
  cbd::GradArgs a;
  std::memset(&a, 0, sizeof(a));
  a.partial = (double*)ws;
  a.norm = norm;
  a.max_norm = max_norm;
  a.partials = plan->partials;
  int err = 0;
  auto fill = [&](const cbd::GradBatch& b) {
    for (int32_t j = 0; j < b.n; j++) {
      const int32_t i = plan->index[b.begin + j];
      a.t[j] = {grads[i], outs ? outs[i] : const_cast<void*>(grads[i]), plan->counts[i],
                plan->chunk_begin[b.begin + j], plan->dtypes[i]};
    }
    a.n = b.n;
    a.chunks = b.chunks;
    a.first = b.first;
  };
  const bool small = plan->batches.size() == 1 && plan->batches[0].chunks <= cbd::kGradSmallChunks &&
                     plan->bytes <= (clip ? cbd::kGradSmallClip : cbd::kGradSmallNorm);
  for (const cbd::GradBatch& b : plan->batches) {
    fill(b);
    if (!err) err = small ? cbd::launch_grad_small(a, clip, stream) : cbd::launch_grad_partial(a, b.grid, stream);
  }
  if (small) {
    // done
  } else if (!clip || plan->batches.empty()) {
    if (!err) err = cbd::launch_grad_finish(a, stream);
  } else {
    // Backwards: what the norm read last is still in the caches.
    for (size_t j = plan->batches.size(); j-- > 0;) {
      const cbd::GradBatch& b = plan->batches[j];
      fill(b);
      if (!err) err = cbd::launch_grad_scale(a, b.grid, stream);
    }
  }
  if (err) {
    cbd::set_error(std::string("gradient kernel launch failed: ") + cbd::hip_error_name(err));
    return CBD_ERR_HIP;
  }
  cbd::set_error("");
  return CBD_OK;
}

}  // namespace

extern "C" cbd_status cbd_grad_plan(const int64_t* counts, const int32_t* dtypes, int32_t n,
                                    cbd_grad_plan_t** out_plan) {
  return guarded([&] { return make_plan(counts, dtypes, n, out_plan); });
}

extern "C" void cbd_grad_plan_destroy(cbd_grad_plan_t* plan) { delete plan; }

extern "C" cbd_status cbd_grad_workspace_size(const cbd_grad_plan_t* plan, uint64_t* bytes) {
  return guarded([&]() -> cbd_status {
    if (!plan || !bytes) return fail(CBD_ERR_INVALID_ARG, "NULL plan or output");
    *bytes = ((uint64_t)plan->partials * sizeof(double) + 255) / 256 * 256 + 256;
    return CBD_OK;
  });
}

extern "C" cbd_status cbd_grad_norm(const cbd_grad_plan_t* plan, const void* const* grads, float* norm,
                                    void* workspace, uint64_t workspace_bytes, void* stream) {
  return guarded(
      [&] { return run(plan, grads, nullptr, false, 0.0, norm, workspace, workspace_bytes, stream); });
}

extern "C" cbd_status cbd_grad_clip(const cbd_grad_plan_t* plan, const void* const* grads, void* const* outs,
                                    double max_norm, float* norm, void* workspace, uint64_t workspace_bytes,
                                    void* stream) {
  return guarded(
      [&] { return run(plan, grads, outs, true, max_norm, norm, workspace, workspace_bytes, stream); });
}
