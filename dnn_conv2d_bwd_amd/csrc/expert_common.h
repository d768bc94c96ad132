// expert_common.h -- host helpers that the entry points over expert rows share:
// errors, strided blocks of memory and what they may not overlap.
#pragma once
#include <cstdint>
#include <string>

#include "cbd_internal.h"

namespace cbd {
namespace host {

inline cbd_status fail(cbd_status s, const char* msg) {
  cbd::set_error(msg);
  return s;
}

inline int esize(int dtype) { return dtype == CBD_F32 ? 4 : 2; }

// A 2-D (or, with count > 1, 3-D) strided block of memory.
struct Block {
  const void* p;
  int64_t rows, width, ld;   // elements
  int64_t count, stride;     // slices
  int es;
  uint64_t span() const {
    if (rows <= 0 || count <= 0) return 0;
    return (uint64_t)((count - 1) * stride + (rows - 1) * ld + width) * es;
  }
};

// Whether two blocks share a byte.  Column slices of one buffer (the same row
// pitch, no slices) are told apart; otherwise the whole spans count.
inline bool share(const Block& a, const Block& b) {
  const uint64_t sa = a.span(), sb = b.span();
  if (!sa || !sb) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (!(x < y + sb && y < x + sa)) return false;
  if (a.count == 1 && b.count == 1 && a.ld * a.es == b.ld * b.es) {
    const uint64_t pitch = (uint64_t)a.ld * a.es, wa = (uint64_t)a.width * a.es, wb = (uint64_t)b.width * b.es;
    const uint64_t d = x <= y ? (y - x) % pitch : (pitch - (x - y) % pitch) % pitch;
    if (d >= wa && d + wb <= pitch) return false;
  }
  return true;
}

constexpr int64_t kMaxSlice = int64_t(1) << 31;  // bytes: offsets within a slice or tile are 32-bit

// Threads of a workgroup, and the most workgroups of a launch (a grid has fewer
// than 2^32 threads).
constexpr int kThreads = 256;
constexpr int64_t kMaxGrid = UINT32_MAX / kThreads;

// Whether every row of a block starts on a 16-byte boundary.
inline bool on16(const Block& b) {
  return (((uintptr_t)b.p | (uint64_t)(b.ld * b.es) | (uint64_t)(b.count > 1 ? b.stride * b.es : 0)) & 15u) == 0;
}

// Runs f, turning a C++ exception (the error string's allocation) into a status.
template <typename F>
cbd_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return CBD_ERR_NO_MEMORY;
  }
}

}  // namespace host
}  // namespace cbd
