// kern_grad_norm.hip -- the global gradient norm and clipping.
//
// Pass 1 (grad_partial): a persistent grid of up to 2048 workgroups walks the
// batch's 64 KiB chunks; each thread keeps a 64-bit sum of squares (a widened
// f32 square is exact there and cannot overflow), and each workgroup writes
// one partial.  Pass 2: every workgroup sums all partials in the same order
// (from L2), so they agree on the factor without another launch or an atomic,
// then scales its chunks; or, for the norm alone, one workgroup does.
//
// A batch of 112 tensors leaves up to 16 KiB of partials and every workgroup of
// every batch reads those of all, so this part grows with the square of the
// batches: little up to some hundred tensors, but 5000 of 1.2 MB (45 batches,
// 720 KiB of partials) read 68 GB from the caches to clip 6 GB.
//
// Pass 2 walks the chunks backwards, so that it starts with what the caches
// still hold, and its accesses are non-temporal: neither its inputs nor its
// results are read again (0.54 G f32 elements 1210 -> 1145 us, 120 M mixed
// ones 205 -> 180 us).
//
// Bound: HBM.  The norm reads every element once (1.5 G elements, nine in ten
// bf16, at 5.8 TB/s); clipping reads it again and writes it (5.7 TB/s; a large
// copy reaches 4.8).
#include "cbd_device.h"
#include "grad_internal.h"

namespace cbd {
namespace {

constexpr int THREADS = 256;
constexpr int VEC = 16;  // bytes per lane and load

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Tensors start at any element: 16-byte accesses at 2-byte alignment, which
// the hardware takes at full rate but for the lines touched twice.
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));

// The tensor holding chunk c of the batch (entries ascend by chunk_begin):
// the entries that begin at or before c, counted 64 at a time across lanes.
__device__ inline int find_tensor(const GradArgs& a, uint32_t c) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int i = 0; i < a.n; i += 64) {
    const int j = i + lane;
    n += __popcll(__ballot(j < a.n && a.t[j < a.n ? j : 0].chunk_begin <= c));
  }
  return n - 1;
}

// Sum over a workgroup in a fixed order; valid in every thread.
template <int T>
__device__ inline double block_sum(double v) {
  __shared__ double part[T / 64];
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < T / 64; i++) s += part[i];
  return s;
}

struct Chunk {
  const char* in;
  char* out;
  uint32_t bytes;
  int dtype;
};

__device__ inline Chunk chunk_of(const GradArgs& a, uint32_t c) {
  const GradEntry& t = a.t[__builtin_amdgcn_readfirstlane(find_tensor(a, c))];
  const int64_t off = (int64_t)(c - t.chunk_begin) * kGradChunkBytes;
  const int64_t left = t.count * (t.dtype == CBD_F32 ? 4 : 2) - off;
  return {(const char*)t.in + off, (char*)t.out + off,
          (uint32_t)(left < kGradChunkBytes ? left : kGradChunkBytes), t.dtype};
}

template <bool F32>
__device__ inline void square16(u32x4 v, double (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (F32) {
      const double d = (double)__uint_as_float(v[i]);
      s[i] = __builtin_fma(d, d, s[i]);
    } else {
      const double lo = (double)dev::bf16_to_f32(v[i] & 0xffffu), hi = (double)__uint_as_float(v[i] & 0xffff0000u);
      s[i] = __builtin_fma(lo, lo, s[i]);
      s[i] = __builtin_fma(hi, hi, s[i]);
    }
  }
}

template <bool F32>
__device__ inline void square_chunk(const Chunk& c, uint32_t tid, double (&s)[4]) {
  constexpr int U = 4;
  constexpr uint32_t STEP = THREADS * VEC;
  const uint32_t whole = c.bytes / VEC * VEC;
  uint32_t at = tid * VEC;
  for (; at + (U - 1) * STEP < whole; at += U * STEP) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; u++) v[u] = *(const u32x4u*)(c.in + at + u * STEP);
#pragma unroll
    for (int u = 0; u < U; u++) square16<F32>(v[u], s);
  }
  for (; at < whole; at += STEP) square16<F32>(*(const u32x4u*)(c.in + at), s);
  // Fewer than 16 bytes are left: an element a thread.
  constexpr uint32_t ES = F32 ? 4 : 2;
  const uint32_t e = whole + tid * ES;
  if (e < c.bytes) {
    const double d = F32 ? (double)*(const float*)(c.in + e) : (double)dev::bf16_to_f32(*(const uint16_t*)(c.in + e));
    s[0] = __builtin_fma(d, d, s[0]);
  }
}

__device__ inline void square_chunk(const Chunk& c, uint32_t tid, double (&s)[4]) {
  if (c.dtype == CBD_F32)
    square_chunk<true>(c, tid, s);
  else
    square_chunk<false>(c, tid, s);
}

__global__ __launch_bounds__(THREADS) void grad_partial_kernel(const GradArgs a) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const Chunk k = chunk_of(a, c);
    square_chunk(k, threadIdx.x, s);
  }
  const double t = block_sum<THREADS>((s[0] + s[1]) + (s[2] + s[3]));
  if (threadIdx.x == 0) a.partial[a.first + blockIdx.x] = t;
}

__device__ inline double norm_of(const GradArgs& a) {
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < a.partials; i += THREADS) s += a.partial[i];
  return __builtin_sqrt(block_sum<THREADS>(s));
}

__global__ __launch_bounds__(THREADS) void grad_finish_kernel(const GradArgs a) {
  const double n = norm_of(a);
  if (threadIdx.x == 0) *a.norm = (float)n;
}

// g times the factor in 64 bits (the factor of a norm near f32's limit is a
// subnormal in f32), rounded to f32; bf16 outputs are rounded from there.
__device__ inline float times(float g, double f) { return (float)((double)g * f); }

template <bool F32>
__device__ inline u32x4 scale16(u32x4 v, double f) {
#pragma unroll
  for (int i = 0; i < 4; i++)
    v[i] = F32 ? __float_as_uint(times(__uint_as_float(v[i]), f))
               : dev::bf16_pack2(times(dev::bf16_to_f32(v[i] & 0xffffu), f), times(__uint_as_float(v[i] & 0xffff0000u), f));
  return v;
}

template <bool F32>
__device__ inline void scale_chunk(const Chunk& c, uint32_t tid, double f) {
  constexpr int U = 4;
  constexpr uint32_t STEP = THREADS * VEC;
  const uint32_t whole = c.bytes / VEC * VEC;
  uint32_t at = tid * VEC;
  for (; at + (U - 1) * STEP < whole; at += U * STEP) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; u++) v[u] = __builtin_nontemporal_load((const u32x4u*)(c.in + at + u * STEP));
#pragma unroll
    for (int u = 0; u < U; u++) __builtin_nontemporal_store(scale16<F32>(v[u], f), (u32x4u*)(c.out + at + u * STEP));
  }
  for (; at < whole; at += STEP) *(u32x4u*)(c.out + at) = scale16<F32>(*(const u32x4u*)(c.in + at), f);
  constexpr uint32_t ES = F32 ? 4 : 2;
  const uint32_t e = whole + tid * ES;
  if (e < c.bytes) {
    if (F32)
      *(float*)(c.out + e) = times(*(const float*)(c.in + e), f);
    else
      *(uint16_t*)(c.out + e) = (uint16_t)dev::bf16_rne(times(dev::bf16_to_f32(*(const uint16_t*)(c.in + e)), f));
  }
}

__device__ inline void scale_chunk(const Chunk& c, uint32_t tid, double f) {
  if (f == 1.0 && c.in == c.out) return;  // g * 1 is g
  if (c.dtype == CBD_F32)
    scale_chunk<true>(c, tid, f);
  else
    scale_chunk<false>(c, tid, f);
}

// By comparison, so that a NaN norm gives a NaN factor.
__device__ inline double factor_of(const GradArgs& a, double n) {
  const double r = a.max_norm / (n + 1e-6);
  return r > 1.0 ? 1.0 : r;
}

__global__ __launch_bounds__(THREADS) void grad_scale_kernel(const GradArgs a) {
  const double n = norm_of(a);
  const double f = factor_of(a, n);
  if (a.first == 0 && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)n;
  for (uint32_t i = blockIdx.x; i < a.chunks; i += gridDim.x) {
    const Chunk k = chunk_of(a, a.chunks - 1 - i);
    scale_chunk(k, threadIdx.x, f);
  }
}

// A list of few chunks: norm and, with clip, scaling by one workgroup, in one
// launch; four waves a chunk.
constexpr int SMALL_THREADS = 1024;
__global__ __launch_bounds__(SMALL_THREADS) void grad_small_kernel(const GradArgs a, int clip) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const uint32_t group = threadIdx.x / THREADS, tid = threadIdx.x % THREADS;
  for (uint32_t c = group; c < a.chunks; c += SMALL_THREADS / THREADS) square_chunk(chunk_of(a, c), tid, s);
  const double n = __builtin_sqrt(block_sum<SMALL_THREADS>((s[0] + s[1]) + (s[2] + s[3])));
  if (threadIdx.x == 0) *a.norm = (float)n;
  if (!clip) return;
  const double f = factor_of(a, n);
  for (uint32_t c = group; c < a.chunks; c += SMALL_THREADS / THREADS) scale_chunk(chunk_of(a, c), tid, f);
}

int launch(const void* k, const GradArgs& a, uint32_t grid, void* stream) {
  void* args[] = {const_cast<GradArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3(grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace

int launch_grad_partial(const GradArgs& a, uint32_t grid, void* stream) {
  return launch((const void*)&grad_partial_kernel, a, grid, stream);
}
int launch_grad_finish(const GradArgs& a, void* stream) {
  return launch((const void*)&grad_finish_kernel, a, 1, stream);
}
int launch_grad_small(const GradArgs& a, int clip, void* stream) {
  void* args[] = {const_cast<GradArgs*>(&a), &clip};
  return (int)hipLaunchKernel((const void*)&grad_small_kernel, dim3(1), dim3(SMALL_THREADS), args, 0,
                              (hipStream_t)stream);
}
int launch_grad_scale(const GradArgs& a, uint32_t grid, void* stream) {
  return launch((const void*)&grad_scale_kernel, a, grid, stream);
}

}  // namespace cbd
