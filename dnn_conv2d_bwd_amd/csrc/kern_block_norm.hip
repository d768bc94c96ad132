// kern_block_norm.hip -- the norms around a block, with its gate and residual.
//
//   yn = y * ry,  ry = 1 / sqrt(mean y^2 + eps)      (y itself where it is not normed)
//   z  = r + scale * gate * w_post * yn
//   zn = z * rz,  rz = 1 / sqrt(mean z^2 + eps),     n = w_pre * zn
//
// Backward, with v = w_pre * dn and c = scale * gate * w_post:
//   dz' = dz + rz * (v - zn * S1 / C)                S1 = sum v * zn
//   dr = dz',  q = c * dz',  dy = ry * (q - yn * S2 / C),  S2 = sum q * yn
// S2 = sum c * yn * (dz + rz * v) - rz * S1 / C * sum c * yn * zn, so that the
// three sums of a row come from one round over its threads.  The vectors'
// gradients need sum dn * zn and sum scale * dz' * yn over the rows: w_post and
// a gate vector are factors of the second that a column shares.  Without dn the
// second norm takes no part (w_pre is NULL then): what r and w_pre hold, which may
// be infinite, reaches nothing.
//
// A row stays in registers from its one load to its stores, 16 bytes a thread: a
// workgroup (or, up to 64 threads a row, a part of one) takes rows i, i + grid,
// ..., loads the next one before it joins the sums of this one, and keeps its
// columns' sums in registers for 128 rows, then adds them up in LDS; in the end they
// go to memory, one row of them a workgroup, for a second launch to join in a fixed
// order.  z is rounded where it is stored, not where n is made of it.
//
// Bound: HBM.  32768 x 4096 in bf16, vectors for all three: forward 212 us (5.1
// TB/s; a copy on this card reaches 4.7), backward 302 (5.3) and 5 for the
// joining; 65536 x 1024 94 and 165, 65536 x 128 13.4 and 20 (67 and 100 MB: the
// caches hold a part); in f32 8192 x 2048 45 and 79.  Of 250 MB, other widths from 72
// to 8192 reach 3.9 - 5.4 TB/s forward and 4.2 - 5.5 backward, the least just
// above a power of two, where half the threads have nothing.  With all sums through
// LDS and the vectors held as f32, rows of 4096 took 393 us backward.  One row: 3
// us, one round to memory and two sums over the waves.
#include <type_traits>

#include "block_internal.h"
#include "cbd_device.h"

namespace cbd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));

// A 16-byte chunk of a row, as it lies in memory.
template <typename T>
struct Chunk {
  static constexpr int N = 16 / sizeof(T);
  using any = std::conditional_t<sizeof(T) == 4, u32x4_4, u32x4_2>;
  u32x4 v;
  __device__ inline void zero() { v = u32x4{0u, 0u, 0u, 0u}; }
  // The first n of its elements (n <= 0: none) from p, zeros after them.
  __device__ inline void load(const T* p, int n) {
    if (n >= N) {
      v = *(const any*)p;
      return;
    }
    zero();
#pragma unroll
    for (int j = 0; j < N - 1; j++)
      if (j < n) {
        if constexpr (sizeof(T) == 4)
          v[j] = ((const uint32_t*)p)[j];
        else
          v[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
      }
  }
  __device__ inline void store(T* p, int n) const {
    if (n >= N) {
      *(any*)p = v;
      return;
    }
#pragma unroll
    for (int j = 0; j < N - 1; j++)
      if (j < n) {
        if constexpr (sizeof(T) == 4)
          ((uint32_t*)p)[j] = v[j];
        else
          p[j] = (T)(v[j >> 1] >> (16 * (j & 1)));
      }
  }
  __device__ inline float get(int j) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(v[j]);
    else
      return j & 1 ? __uint_as_float(v[j >> 1] & 0xffff0000u) : __uint_as_float(v[j >> 1] << 16);
  }
  __device__ inline void put(const float (&f)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] = __float_as_uint(f[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] = dev::bf16_pack2(f[2 * j], f[2 * j + 1]);
    }
  }
};

// v and its partner's, LANES / 2 lanes away or mirrored: after all steps every
// lane of a group of LANES (a power of two up to 64) has the group's sum, each
// with the same bits, since the two of a step add the same two values.
template <int CTRL>
__device__ inline float plus_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int LANES>
__device__ inline float group_sum(float v) {
  if constexpr (LANES >= 2) v = plus_dpp<0xb1>(v);    // quad_perm 1 0 3 2
  if constexpr (LANES >= 4) v = plus_dpp<0x4e>(v);    // quad_perm 2 3 0 1
  if constexpr (LANES >= 8) v = plus_dpp<0x141>(v);   // row_half_mirror
  if constexpr (LANES >= 16) v = plus_dpp<0x140>(v);  // row_mirror
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16, 64);
  if constexpr (LANES >= 64) v += __shfl_xor(v, 32, 64);
  return v;
}

// Sums over a row's threads, in a fixed order, for everyone.  Two buffers, so
// that one barrier is enough: who writes a buffer again has passed the other's
// barrier, before which everyone has read it.
template <int LANES, int S>
struct RowSum {
  static constexpr int W = LANES > 64 ? LANES / 64 : 1;
  float (*part)[S][W];
  int at = 0;
  __device__ inline void operator()(float (&s)[S]) {
#pragma unroll
    for (int i = 0; i < S; i++) s[i] = group_sum<LANES < 64 ? LANES : 64>(s[i]);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < S; i++) part[at][i][threadIdx.x >> 6] = s[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < S; i++) s[i] = group_sum<W>(part[at][i][threadIdx.x & (W - 1)]);
      at ^= 1;
    }
  }
};

// Opaque to the compiler, which would keep vectors widened to f32 through the
// loop over rows: twice the registers.
template <typename T, int CH>
__device__ inline void as_loaded(Chunk<T> (&v)[CH]) {
#pragma unroll
  for (int i = 0; i < CH; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t w = v[i].v[j];
      asm volatile("" : "+v"(w));
      v[i].v[j] = w;
    }
}

template <int LANES>
constexpr int kThreads = LANES <= 64 ? 256 : LANES;
// Waves a SIMD: 128 registers (1024 threads have no more) where a thread has
// one chunk; with rows inside a wave, whose addresses take registers, 168.
template <int LANES, int CH>
constexpr int kWaves = CH > 1 ? 1 : LANES < 64 ? 3 : 4;
// The next row is loaded ahead; with more chunks a thread has no room for it.
template <int CH>
constexpr bool kAhead = CH == 1;
// Backward, a thread with more than 8 elements a row has no room for what both
// rounds over the row need, nor for its columns' sums: it reads its chunks again
// in the second one, and keeps the sums in LDS (4096 rows of 10240 in
// bf16 166 us, held, with spills, 484; of 16384 224 / 503; 2048 rows of 16384 in
// f32 300 / 495; 4096 of 8192, which fit, 161 held and 211 read again).
template <typename T, int CH>
constexpr bool kHeld = block_held(CH, sizeof(T));

// What a thread has of its rows: CH chunks, LANES chunks apart.
template <typename T, int LANES, int CH>
struct Rows {
  static constexpr int N = Chunk<T>::N;
  int lane, n[CH];  // elements of each chunk that are inside (negative: none)
  int64_t row, step;
  __device__ inline explicit Rows(const BlockArgs& a) {
    lane = threadIdx.x & (LANES - 1);
#pragma unroll
    for (int i = 0; i < CH; i++) n[i] = a.c - N * (lane + LANES * i);
    constexpr int per = kThreads<LANES> / LANES;
    int sub = threadIdx.x / LANES;
    if (LANES >= 64) sub = __builtin_amdgcn_readfirstlane(sub);
    row = (int64_t)blockIdx.x * per + sub;
    step = (int64_t)gridDim.x * per;
  }
  __device__ inline void load(Chunk<T>& v, const void* p, int64_t at, int i) const {
    v.load((const T*)p + at + N * (lane + LANES * i), n[i]);
  }
  __device__ inline void load(Chunk<T> (&v)[CH], const void* p, int64_t at) const {
#pragma unroll
    for (int i = 0; i < CH; i++) load(v[i], p, at, i);
  }
  __device__ inline void store(const Chunk<T>& v, void* p, int64_t at, int i) const {
    v.store((T*)p + at + N * (lane + LANES * i), n[i]);
  }
  __device__ inline void store(const Chunk<T> (&v)[CH], void* p, int64_t at) const {
#pragma unroll
    for (int i = 0; i < CH; i++) store(v[i], p, at, i);
  }
  __device__ inline static void zero(Chunk<T> (&v)[CH]) {
#pragma unroll
    for (int i = 0; i < CH; i++) v[i].zero();
  }
  // A vector, or ones in its place: factors that change nothing.
  __device__ inline void vector(Chunk<T>& v, const void* p, int i) const {
    constexpr uint32_t one = sizeof(T) == 4 ? 0x3f800000u : 0x3f803f80u;
    if (p)
      load(v, p, 0, i);
    else
      v.v = u32x4{one, one, one, one};
  }
  __device__ inline void vector(Chunk<T> (&v)[CH], const void* p) const {
#pragma unroll
    for (int i = 0; i < CH; i++) vector(v[i], p, i);
  }
};

__device__ inline float inverse_rms(float squares, const BlockArgs& a) {
  return 1.f / __builtin_sqrtf(squares / (float)a.c + a.eps);
}

template <typename T, int LANES, int CH>
__global__ __launch_bounds__(kThreads<LANES>, (kWaves<LANES, CH>)) void block_forward_kernel(const BlockArgs a) {
  constexpr int N = Chunk<T>::N;
  __shared__ float part[2][1][RowSum<LANES, 1>::W];
  RowSum<LANES, 1> sum{part};
  Rows<T, LANES, CH> rows(a);
  Chunk<T> wq[CH], gq[CH], wp[CH];  // w_post, gate, w_pre
  rows.vector(wq, a.w_post);
  rows.vector(gq, a.gate_rows ? nullptr : a.gate);
  rows.vector(wp, a.w_pre);
  Chunk<T> r[CH], y[CH], g[CH];
  Rows<T, LANES, CH>::zero(y);
  auto fetch = [&](int64_t row) {
    rows.load(r, a.r, row * a.ldr);
    if (a.y) rows.load(y, a.y, row * a.ldy);
    if (a.gate_rows) rows.load(g, a.gate, row * a.ldgate);
  };
  if (kAhead<CH> && rows.row < a.rows) fetch(rows.row);
  for (int64_t row = rows.row; row < a.rows; row += rows.step) {
    if (!kAhead<CH>) fetch(row);
    as_loaded(wq);
    as_loaded(gq);
    as_loaded(wp);
    float z[CH][N], v[CH][N];
#pragma unroll
    for (int i = 0; i < CH; i++)
#pragma unroll
      for (int j = 0; j < N; j++) {
        z[i][j] = r[i].get(j);
        v[i][j] = y[i].get(j);
      }
    float s[1] = {0.f};
    // What the gate, the weight and the scale make of y.
    Chunk<T> gr[CH];
#pragma unroll
    for (int i = 0; i < CH; i++) gr[i] = a.gate_rows ? g[i] : gq[i];
    if (kAhead<CH> && row + rows.step < a.rows) fetch(row + rows.step);
    float ry = 1.f, rz = 1.f;
    if (a.w_post) {
#pragma unroll
      for (int i = 0; i < CH; i++)
#pragma unroll
        for (int j = 0; j < N; j++) s[0] = __builtin_fmaf(v[i][j], v[i][j], s[0]);
      sum(s);
      ry = inverse_rms(s[0], a);
    }
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < CH; i++)
#pragma unroll
      for (int j = 0; j < N; j++) {
        z[i][j] = __builtin_fmaf(a.scale, v[i][j] * ry * wq[i].get(j) * gr[i].get(j), z[i][j]);
        s[0] = __builtin_fmaf(z[i][j], z[i][j], s[0]);
      }
    if (a.z) {
      Chunk<T> o[CH];
#pragma unroll
      for (int i = 0; i < CH; i++) o[i].put(z[i]);
      rows.store(o, a.z, row * a.ldz);
    }
    if (a.w_pre) {
      sum(s);
      rz = inverse_rms(s[0], a);
      Chunk<T> o[CH];
#pragma unroll
      for (int i = 0; i < CH; i++) {
        float f[N];
#pragma unroll
        for (int j = 0; j < N; j++) f[j] = z[i][j] * rz * wp[i].get(j);
        o[i].put(f);
      }
      rows.store(o, a.n, row * a.ldn);
    }
    if (a.stats && rows.lane == 0) {
      a.stats[2 * row] = ry;
      a.stats[2 * row + 1] = rz;
    }
  }
}

// The gradients that column col's sum (`which` of the two) makes.
__device__ inline void finish_column(const BlockFinish& a, int which, int col, double s) {
  auto vector = [&](const void* v) {
    return !v ? 1.0 : (double)(a.dtype == CBD_F32 ? ((const float*)v)[col] : dev::bf16_to_f32(((const uint16_t*)v)[col]));
  };
  auto put = [&](void* o, double v) {
    if (!o) return;
    if (a.dw_dtype == CBD_F32)
      ((float*)o)[col] = (float)v;
    else
      ((uint16_t*)o)[col] = (uint16_t)dev::bf16_rne((float)v);
  };
  if (which == 0) {
    put(a.dw_pre, s);
  } else {
    // (No rows: zeros, whatever the vectors hold.)
    put(a.dw_post, a.n ? s * vector(a.gate) : 0.0);
    put(a.dgate, a.n ? s * vector(a.w_post) : 0.0);
  }
}

// SECOND: there is a second norm (a.w_pre), known beforehand.
template <typename T, int LANES, int CH, bool SECOND = false>
__global__ __launch_bounds__(kThreads<LANES>, (kWaves<LANES, CH>)) void block_bwd_kernel(const BlockArgs a) {
  constexpr int N = Chunk<T>::N;
  const bool second = SECOND || a.w_pre;
  constexpr bool HELD = kHeld<T, CH>;
  __shared__ float part[2][3][RowSum<LANES, 3>::W];
  RowSum<LANES, 3> sum{part};
  Rows<T, LANES, CH> rows(a);
  Chunk<T> wq[CH], gq[CH], wp[CH];
  if (HELD) {
    rows.vector(wq, a.w_post);
    rows.vector(gq, a.gate_rows ? nullptr : a.gate);
    rows.vector(wp, a.w_pre);
  }
  // The columns' sums.
  __shared__ f32x4 sums[HELD ? 1 : 2 * CH * N / 4][HELD ? 1 : kThreads<LANES>];
  float pre[CH][N], post[CH][N];
  // Takes in (out of) registers what LDS has of chunk i.
  auto take = [&](float (&v)[N], int at) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const f32x4 q = sums[at * (N / 4) + j / 4][threadIdx.x];
#pragma unroll
      for (int k = 0; k < 4; k++) v[j + k] = q[k];
    }
  };
  auto leave = [&](const float (&v)[N], int at) {
#pragma unroll
    for (int j = 0; j < N; j += 4) sums[at * (N / 4) + j / 4][threadIdx.x] = f32x4{v[j], v[j + 1], v[j + 2], v[j + 3]};
  };
#pragma unroll
  for (int i = 0; i < CH; i++) {
#pragma unroll
    for (int j = 0; j < N; j++) pre[i][j] = post[i][j] = 0.f;
    if (!HELD) {
      leave(pre[i], i);
      leave(post[i], CH + i);
    }
  }
  // No second norm or no dn: dw_pre is 0, not the sum of 0 times what r holds.
  auto first = [&](int i, int j) { return second ? pre[i][j] : 0.f; };
  // The columns' sums go on to LDS and begin again after every kBlockJoin rows: one f32
  // sum of many rows would lose what is small next to all of them.  (Where LDS holds
  // the sums themselves the plan has a workgroup for as many rows.)
  float* const out = a.partial + (int64_t)blockIdx.x * 2 * a.c;
  __shared__ float join[2][HELD ? CH * N : 1][HELD ? kThreads<LANES> : 1];
  int since = 0;
  bool more = false;
  auto pass_on = [&]() {
    int tid = LANES > 64 ? rows.lane : (int)threadIdx.x;
    asm volatile("" : "+v"(tid));  // no addresses in registers through the loop over rows
#pragma unroll
    for (int i = 0; i < CH; i++)
#pragma unroll
      for (int j = 0; j < N; j++) {
        float &u = join[0][i * N + j][tid], &v = join[1][i * N + j][tid];
        u = more ? u + first(i, j) : first(i, j);
        v = more ? v + post[i][j] : post[i][j];
        pre[i][j] = post[i][j] = 0.f;
      }
    more = true;
    since = 0;
  };
  Chunk<T> r[CH], y[CH], g[CH], dz[CH], dn[CH];
  float ry1 = 1.f, rz1 = 1.f;
  Rows<T, LANES, CH>::zero(y);
  Rows<T, LANES, CH>::zero(dz);
  Rows<T, LANES, CH>::zero(dn);
  auto fetch = [&](int64_t row, int i) {
    rows.load(r[i], a.r, row * a.ldr, i);
    if (a.y) rows.load(y[i], a.y, row * a.ldy, i);
    if (a.dz) rows.load(dz[i], a.dz, row * a.lddz, i);
    if (SECOND || a.dn) rows.load(dn[i], a.dn, row * a.lddn, i);
    if (a.gate_rows) rows.load(g[i], a.gate, row * a.ldgate, i);
  };
  auto statistics = [&](int64_t row) {
    if (a.w_post) ry1 = a.stats[2 * row];
    if (second) rz1 = a.stats[2 * row + 1];
  };
  auto fetch_all = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; i++) fetch(row, i);
    statistics(row);
  };
  if (kAhead<CH> && rows.row < a.rows) fetch_all(rows.row);
  const float inv_c = 1.f / (float)a.c;
  for (int64_t row = rows.row; row < a.rows; row += rows.step) {
    if (!HELD)
      statistics(row);
    else if (!kAhead<CH>)
      fetch_all(row);
    const float ry = ry1, rz = rz1;
    if (HELD) {
      as_loaded(wq);
      as_loaded(gq);
      as_loaded(wp);
    }
    float zn[CH][N], yn[CH][N], e[CH][N];
    Chunk<T> gr[CH];
    float s[3] = {0.f, 0.f, 0.f};
    // Chunk i of zn, yn and e; in the first round over the row also the sums.
    auto chunk = [&](int i, bool sums) {
      if (!HELD) {
        y[i].zero();
        dz[i].zero();
        dn[i].zero();
        g[i].zero();
        fetch(row, i);
        rows.vector(wq[i], a.w_post, i);
        rows.vector(gq[i], a.gate_rows ? nullptr : a.gate, i);
        rows.vector(wp[i], a.w_pre, i);
      }
      gr[i] = a.gate_rows ? g[i] : gq[i];
#pragma unroll
      for (int j = 0; j < N; j++) {
        const float d = dn[i].get(j);
        yn[i][j] = y[i].get(j) * ry;
        const float cy = a.scale * wq[i].get(j) * gr[i].get(j) * yn[i][j];
        zn[i][j] = (r[i].get(j) + cy) * rz;
        const float v = d * wp[i].get(j);
        e[i][j] = __builtin_fmaf(rz, v, dz[i].get(j));
        if (!sums) continue;
        pre[i][j] = __builtin_fmaf(d, zn[i][j], pre[i][j]);
        s[0] = __builtin_fmaf(v, zn[i][j], s[0]);
        s[1] = __builtin_fmaf(cy, e[i][j], s[1]);
        s[2] = __builtin_fmaf(cy, zn[i][j], s[2]);
      }
    };
#pragma unroll
    for (int i = 0; i < CH; i++) {
      if (!HELD) take(pre[i], i);
      chunk(i, true);
      if (!HELD) leave(pre[i], i);
      if (!HELD) __builtin_amdgcn_sched_barrier(0);
    }
    if (kAhead<CH> && row + rows.step < a.rows) fetch_all(row + rows.step);
    sum(s);
    // (Where there is no norm, nothing is taken off: not 0 times infinity.)
    const float along = second ? rz * s[0] * inv_c : 0.f;               // of zn in dz'
    const float back = (second ? s[1] - along * s[2] : s[1]) * inv_c;  // of yn in dy
#pragma unroll
    for (int i = 0; i < CH; i++) {
      if (!HELD) {
        chunk(i, false);
        take(post[i], CH + i);
      }
      Chunk<T> o_r, o_y, o_g;
      float fr[N], fy[N], fg[N];
#pragma unroll
      for (int j = 0; j < N; j++) {
        fr[j] = second ? __builtin_fmaf(-along, zn[i][j], e[i][j]) : e[i][j];
        const float da = a.scale * fr[j], dg = da * gr[i].get(j), w = wq[i].get(j);
        fg[j] = da * yn[i][j] * w;
        post[i][j] = __builtin_fmaf(a.gate_rows ? dg : da, yn[i][j], post[i][j]);
        fy[j] = a.w_post ? ry * __builtin_fmaf(-back, yn[i][j], dg * w) : dg;
      }
      if (!HELD) leave(post[i], CH + i);
      o_r.put(fr);
      o_y.put(fy);
      o_g.put(fg);
      if (a.dr) rows.store(o_r, a.dr, row * a.lddr, i);
      if (a.dy) rows.store(o_y, a.dy, row * a.lddy, i);
      if (a.dgate) rows.store(o_g, a.dgate, row * a.lddgate, i);
      if (!HELD) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (HELD)
      if (++since == kBlockJoin && a.partial) pass_on();
  }
  const bool alone = gridDim.x == 1;  // no one to join
  if (!a.partial) return;
  if constexpr (LANES <= 64) {
    pass_on();
    // The groups' sums, joined in their order.
    constexpr int G = 256 / LANES, COLS = LANES * CH * N;
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * COLS; k += 256) {
      const int which = k / COLS, col = k % COLS, i = col / (N * LANES), lane = col / N % LANES, j = col % N;
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < G; g++) s += join[which][i * N + j][g * LANES + lane];
      if (col < a.c) {
        if (alone)
          finish_column(a.finish, which, col, s);
        else
          out[which * a.c + col] = s;
      }
    }
  } else {
    int lane = rows.lane;
    asm volatile("" : "+v"(lane));  // (as above)
#pragma unroll
    for (int i = 0; i < CH; i++) {
      const int at = N * (lane + LANES * i);
      if (!HELD) {
        take(pre[i], i);
        take(post[i], CH + i);
      }
#pragma unroll
      for (int j = 0; j < N; j++)
        if (at + j < a.c) {
          float u = first(i, j), v = post[i][j];
          if (HELD && more) {
            u += join[0][HELD ? i * N + j : 0][lane];
            v += join[1][HELD ? i * N + j : 0][lane];
          }
          if (alone) {
            finish_column(a.finish, 0, at + j, u);
            finish_column(a.finish, 1, at + j, v);
          } else {
            out[at + j] = u;
            out[a.c + at + j] = v;
          }
        }
    }
  }
}

// 64 columns by 16 slices of the workgroups' sums, which are joined in 64 bits.
constexpr int FINISH = 1024;
__global__ __launch_bounds__(FINISH) void block_finish_kernel(const BlockFinish a) {
  __shared__ double part[FINISH / 64][64];
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane, which = blockIdx.y;
  double s = 0.0;
  if (col < a.c) {
    const float* p = a.partial + (int64_t)which * a.c + col;
#pragma unroll 8
    for (int i = slice; i < a.n; i += FINISH / 64) s += (double)p[(int64_t)i * 2 * a.c];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice > 0 || col >= a.c) return;
#pragma unroll
  for (int i = 1; i < FINISH / 64; i++) s += part[i][lane];
  finish_column(a, which, col, s);
}

template <typename T, bool BWD>
const void* pick(BlockShape s, bool second) {
  constexpr int F = sizeof(T) / 2;
  // bf16 rows that are read twice, which are short of registers, with a second norm:
  // 4096 x 10240 166 us, with the question left open 172 (f32, 2048 x 16384, which
  // spills: 318 / 308).
  if constexpr (BWD && F == 1)
    if (second && !block_held(s.chunks, sizeof(T))) return (const void*)&block_bwd_kernel<T, 1024, 2, true>;
#define CBD_BLOCK(L, C) \
  if (s.lanes == L && s.chunks == C) return BWD ? (const void*)&block_bwd_kernel<T, L, C> : (const void*)&block_forward_kernel<T, L, C>;
  CBD_BLOCK(8, 1)
  CBD_BLOCK(16, 1)
  CBD_BLOCK(32, 1)
  CBD_BLOCK(64, 1)
  CBD_BLOCK(128, 1)
  CBD_BLOCK(256, 1)
  CBD_BLOCK(512, 1)
  CBD_BLOCK(1024, 1)
  CBD_BLOCK(1024, 2)
  if constexpr (F == 2) {
    CBD_BLOCK(1024, 4)
  }
#undef CBD_BLOCK
  return nullptr;
}

template <bool BWD>
int launch(const BlockArgs& a, BlockShape s, int dtype, int64_t grid, void* stream) {
  const void* k = dtype == CBD_F32 ? pick<float, BWD>(s, a.w_pre) : pick<uint16_t, BWD>(s, a.w_pre);
  void* args[] = {const_cast<BlockArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)grid), dim3(block_threads(s)), args, 0,
                              (hipStream_t)stream);
}

}  // namespace

int launch_block_forward(const BlockArgs& a, BlockShape s, int dtype, int64_t grid, void* stream) {
  return launch<false>(a, s, dtype, grid, stream);
}
int launch_block_bwd(const BlockArgs& a, BlockShape s, int dtype, int64_t grid, void* stream) {
  return launch<true>(a, s, dtype, grid, stream);
}
int launch_block_finish(const BlockFinish& a, void* stream) {
  void* args[] = {const_cast<BlockFinish*>(&a)};
  return (int)hipLaunchKernel((const void*)&block_finish_kernel, dim3((unsigned)((a.c + 63) / 64), 2), dim3(FINISH),
                              args, 0, (hipStream_t)stream);
}

}  // namespace cbd
