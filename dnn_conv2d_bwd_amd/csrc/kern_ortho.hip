// kern_ortho.hip -- orthogonalised updates: Newton-Schulz steps
//
//   A = X X^T,  B = a I + b A + c A A,  X <- B X
//
// on matrices held as two halves a value (ortho_internal.h).  A product of two
// such values is hi hi + hi lo + lo hi, three matrix instructions on halves with
// f32 sums; lo lo is below 2^-22 of it.  A value keeps 22 bits: each step's
// rounding is some 2^-24 of it, next to sums of f32 products, whose own are
// larger; and halves go at 16 times the rate of the f32 instructions, so that
// three of them are 5 times as fast.
//
// One exponent a matrix, chosen by the plan from the bounds of the singular values,
// keeps the largest value at 2^14 at most.  Halves end at 2^-24, so small values have
// fewer bits: with lo as it is, those below 2^-3 (2^-17 of the bound).  Rows of 256 x
// 512 that are 1e-6 as large as the others were off by 3.2e-4 then; times 2^11, lo is
// as large as hi, 22 bits reach down to 2^-14, 2^-28 of the bound, and those rows are
// off by 2.8e-7, an f32 form's by 3.5e-7.  The sums of hi lo and lo hi are then 2^11
// times as large as those of hi hi and wait for their own place in registers, or for
// their own turn (TWICE below).
//
// A and B are symmetric: only tiles on and above the diagonal are computed, and
// each is stored twice.  Where A has few of them, workgroups take slices of its
// long side, whose f32 sums a small launch joins.
//
// A workgroup of 4 waves (2 x 2) computes a tile of 64 MB x 64 MB in runs of 32
// k: 128 bytes of a row, hi and lo, go straight to one of NS LDS stages
// (buffer_load ... lds), in chunks of 16 bytes, chunk c of row r at c ^ (r / 2 %
// 8), so that reads of 32 rows spread over the banks.
//
// Bound: large matrices by the matrix instructions, at the rate that the card's
// power allows.  8 x 4096 x 2048 in bf16, a step: A 306 + 79 us (7 matrices in tiles
// of 256, one in tiles of 128 for the units that those leave idle), B 176 + 49, X 675
// (1.22 PFLOP/s of halves; a library product of 8192 x 8192 x 8192 in bf16 reaches
// 1.26), the last 620 (1.33: it writes a quarter of the bytes); five steps with
// norm (31 us, 4.3 TB/s) and split (103, 6.5 TB/s, two directions of 4 bytes
// written) 6.3 - 6.6 ms.  In f32 A 362 + 79, B 198 + 49, X 760, the last 718, 7.3 ms.
// Results leave through LDS in whole columns of blocks: 0.3 ms less than block by
// block.  Small ones by latency: 16 x 256 x 512 takes 7 to 11 us a launch for 8 to 16
// runs.
//
// Stages: one workgroup of 64 x 64 a compute unit waits for every load and LDS
// read, so four runs are in flight and one in registers (5 / 3 / 2 stages: A of
// 1024 x 1024 12 / 26 / 25 us); tiles of 128 likewise while there is one a unit (4
// / 2 stages: 136 tiles of 64 runs 46 / 62 us), two a unit hide each other's ways
// (363 tiles of 44 runs 74 / 55); tiles of 256 have LDS for two stages, and 96
// products a run to hide their loads.  Tiles of 256 that sum twice have 64 products a
// run and more to read for each: five stages of one operand, all of the LDS, where
// each is filled again as soon as it is free, 7.26 ms for 8 x 4096 x 2048 in f32, two
// of both 7.42 (one set of sums for both kinds 6.37); matrix units busy 54 - 64 % of the
// clocks instead of 60 - 78, for half as many LDS reads again and 64-byte lines in the
// second turn.
#include <type_traits>

#include "cbd_device.h"
#include "ortho_internal.h"

namespace cbd {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((__vector_size__(16 * sizeof(float))));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
#define INLINE __attribute__((always_inline))

constexpr int THREADS = 256;

__device__ inline uint16_t half_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ inline float half_value(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }
// The two halves of a value: hi in bits 0-15, lo, `up` times what hi leaves, in
// bits 16-31.
__device__ inline uint32_t split(float v, float up) {
  const uint16_t hi = half_bits(v);
  return hi | (uint32_t)half_bits((v - half_value(hi)) * up) << 16;
}

// s_waitcnt: every load and LDS access is done.
__device__ inline void wait_all() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0 | (7 << 4));  // vmcnt 0, expcnt 7, lgkmcnt 0
  asm volatile("" ::: "memory");
}
// And one where up to n loads may be on their way, and (LDS = 15) LDS accesses.
template <int n, int LDS = 15>
__device__ inline void wait_loads() {
  static_assert(n < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (LDS << 8) | ((n >> 4) << 14));
  asm volatile("" ::: "memory");
}
__device__ inline void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Tile (mt, nt), n >= m, of a symmetric matrix of n x n tiles: groups of W columns,
// in each row by row; neighbours, which one XCD has, share both operands.
__device__ inline void upper_tile(int local, int n, int W, int& mt, int& nt) {
  int c0 = 0, w = n < W ? n : W;
  while (local >= c0 * w + w * (w + 1) / 2) {
    local -= c0 * w + w * (w + 1) / 2;
    c0 += w;
    w = n - c0 < W ? n - c0 : W;
  }
  if (local < c0 * w) {
    mt = local / w;
    nt = c0 + local - mt * w;
  } else {
    local -= c0 * w;
    int r = 0;
    for (; local >= w - r; r++) local -= w - r;
    mt = c0 + r;
    nt = mt + local;
  }
}

template <int MB, int STAGE, int NS, bool TWICE = false>
__global__ __launch_bounds__(THREADS, MB == 4 || (MB == 2 && NS > 2) ? 1 : 2) void ortho_product_kernel(const OrthoArgs a) {
  constexpr int T = 64 * MB;
  constexpr int BYTES = T * 128;      // of an operand's stage
  constexpr int N = BYTES / 4096;     // 1 KiB blocks of it that a wave fills
  constexpr bool SLICE = STAGE == ORTHO_SLICE, SYM = STAGE == ORTHO_SQUARE || STAGE == ORTHO_POLY || SLICE;
  __shared__ __attribute__((aligned(1024))) char smem[TWICE ? 5 * BYTES : 2 * NS * BYTES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;

  // The matrix and the tile.
  const int per = SYM ? a.tiles_m * (a.tiles_m + 1) / 2 : a.tiles_m * a.tiles_n;
  const int block = dev::logical_tile((int)blockIdx.x, (int)gridDim.x, 1), t = SLICE ? block / a.slices : block;
  const int run0 = SLICE ? __builtin_amdgcn_readfirstlane((block - t * a.slices) * a.slice) : 0;
  const int runs = SLICE && a.runs - run0 > a.slice ? a.slice : a.runs - run0;
  const int mat = __builtin_amdgcn_readfirstlane(t / per);
  int local = __builtin_amdgcn_readfirstlane(t - mat * per), mt, nt;
  if (SYM) {
    upper_tile(local, a.tiles_n, gridDim.x <= 256 ? 4 : 8, mt, nt);
  } else {
    // Groups of 8 rows of tiles by all columns.
    const int g = local / (8 * a.tiles_n), in = local - g * 8 * a.tiles_n;
    const int gm = a.tiles_m - 8 * g < 8 ? a.tiles_m - 8 * g : 8;
    nt = in / gm;
    mt = 8 * g + in - nt * gm;
  }
  mt = __builtin_amdgcn_readfirstlane(mt);
  nt = __builtin_amdgcn_readfirstlane(nt);

  // ORTHO_POLY: A itself, where it will be added (it is symmetric: row `col` has
  // four neighbouring elements of a lane).  Tiles of 256 have no registers for it
  // until the sums are done.
  constexpr bool EARLY = STAGE == ORTHO_POLY && MB < 4;
  u32x2 own[EARLY ? MB * MB : 1][8];
  auto fetch = [&](int m, int n, u32x2 (&o)[8]) INLINE {
    const int col = T * nt + 32 * MB * wn + 32 * n + (lane & 31), run = ((T * mt + 32 * MB * wm) >> 5) + m;
    const uint16_t* d = a.p + mat * a.p_mat + (int64_t)col * a.ldp + run * 64 + 4 * (lane >> 5);
#pragma unroll
    for (int q = 0; q < 4; q++) {
      o[q] = *(const u32x2*)(d + 8 * q);
      o[4 + q] = *(const u32x2*)(d + 8 * q + 32);
    }
  };
  if constexpr (EARLY) {
#pragma unroll
    for (int n = 0; n < MB; n++)
#pragma unroll
      for (int m = 0; m < MB; m++) fetch(m, n, own[n * MB + m]);
  }

  // Loads: row lane / 8 of every 8, chunk lane % 8 in LDS.
  uint64_t bp = (uint64_t)(a.p + mat * a.p_mat + (int64_t)mt * T * a.ldp + run0 * 64);
  uint64_t bq = (uint64_t)(a.q + mat * a.q_mat + (int64_t)nt * T * a.ldq + run0 * 64);
  uint32_t vp[N], vq[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int row = 8 * (N * wave + i) + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
    vp[i] = (uint32_t)row * (uint32_t)a.ldp * 2u + (uint32_t)c * 16u;
    vq[i] = (uint32_t)row * (uint32_t)a.ldq * 2u + (uint32_t)c * 16u;
  }
  const uint32_t rec_p = (uint32_t)T * (uint32_t)a.ldp * 2u, rec_q = (uint32_t)T * (uint32_t)a.ldq * 2u;
  const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char*)smem + (uint32_t)(wave * N * 1024));
  auto issue = [&](uint64_t b, uint32_t rec, uint32_t voff, uint32_t soff, uint32_t m0v) INLINE {
    const i32x4 d = {(int)(uint32_t)b, (int)((uint32_t)(b >> 32) & 0xffffu), (int)rec, 0x00020000};
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds\n\ts_nop 0"
                 ::"s"(m0v), "v"(voff), "s"(d), "s"(soff) : "memory", "m0");
#pragma clang diagnostic pop
  };
  // Run k of an operand into stage s; past the last there is nothing to load
  // (a record count of 0 gives zeros), but the count of loads stays.
  auto load_p = [&](int k, int s, int i) INLINE {
    issue(bp, k < runs ? rec_p : 0u, vp[i], (uint32_t)k * 128u, base + (uint32_t)(2 * s * BYTES + i * 1024));
  };
  auto load_q = [&](int k, int s, int i) INLINE {
    issue(bq, k < runs ? rec_q : 0u, vq[i], (uint32_t)k * 128u, base + (uint32_t)((2 * s + 1) * BYTES + i * 1024));
  };
  // The same where after the runs come their hi alone, 64 of them at a time: chunks
  // 4 .. 7 of a row are then those of the next run, 64 bytes further on than its lo.
  // (c / 4 of the chunks above, with N * wave even.)
  const int doubles = (runs + 1) / 2;
  [[maybe_unused]] const uint32_t further[2] = {(uint32_t)(lane & 4) << 4, (uint32_t)(~lane & 4) << 4};
  [[maybe_unused]] auto load_twice = [&](uint64_t b, uint32_t rec, uint32_t voff, int k, int i, uint32_t m0v) INLINE {
    const int h = k - runs;
    issue(b, h < doubles ? rec : 0u, voff + (h < 0 ? 0u : further[i & 1]), (uint32_t)(h < 0 ? k * 128 : h * 256), m0v);
  };

  // Fragments: 32 rows by 16 k; half h (0: hi, 1: lo) of k 16 ks ...
  int at_p[4], at_q[4];
  {
    const int rp = 32 * MB * wm + (lane & 31), rq = 32 * MB * wn + (lane & 31);
#pragma unroll
    for (int c = 0; c < 4; c++) {
      at_p[c] = rp * 128 + (((2 * c + (lane >> 5)) ^ ((rp >> 1) & 7)) << 4);
      at_q[c] = rq * 128 + (((2 * c + (lane >> 5)) ^ ((rq >> 1) & 7)) << 4);
    }
  }
  auto read_p = [&](int s, int ks, int h, int b) INLINE {
    return *(const f16x8*)(smem + 2 * s * BYTES + at_p[2 * h + ks] + b * 4096);
  };
  auto read_q = [&](int s, int ks, int h, int b) INLINE {
    return *(const f16x8*)(smem + (2 * s + 1) * BYTES + at_q[2 * h + ks] + b * 4096);
  };

  // Sums of hi hi and, apart where registers allow it, of hi lo and lo hi: these
  // are 2^-11 of the others, and so are their roundings then (3 steps of 9 matrices
  // of 512 x 768 are off by 1.15e-6 together, 0.73e-6 apart; an f32 library product's
  // form by 0.85e-6).  Tiles of 256 have registers for one set: they join the two
  // kinds (lo_up is 1 then) or sum them one after the other (TWICE).
  constexpr bool APART = MB < 4;
  f32x16 acc[MB][MB], low[APART ? MB : 1][APART ? MB : 1];

  // MFMAs on (x, y), with R reads and L loads spread between them.
  const f32x16 zero = {};
  // first: the sums begin.  hi: these are hi hi.
  auto multiply = [&](bool first, bool hi, int m, int n, const f16x8& x, const f16x8& y) INLINE {
    f32x16& sum = APART && !hi ? low[APART ? m : 0][APART ? n : 0] : acc[m][n];
    sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, first ? zero : sum, 0, 0, 0);
  };
  auto part = [&](auto firstc, auto hic, const f16x8 (&x)[MB], const f16x8 (&y)[MB], auto rc, auto&& rd, auto lc,
                  auto&& ld) INLINE {
    constexpr int Q = MB * MB, R = decltype(rc)::value, L = decltype(lc)::value;
#pragma unroll
    for (int i = 0; i < Q; i++) {
      const int n = i / MB, m = (n & 1) ? MB - 1 - i % MB : i % MB;
      multiply(firstc.value, hic.value, m, n, x[m], y[n]);
#pragma unroll
      for (int r = i * R / Q; r < (i + 1) * R / Q; r++) rd(r);
#pragma unroll
      for (int r = i * L / Q; r < (i + 1) * L / Q; r++) ld(r);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  constexpr std::true_type hi{};
  constexpr std::false_type lo{};
  constexpr std::integral_constant<int, 0> none{};
  constexpr std::integral_constant<int, MB> one{};
  constexpr std::integral_constant<int, 2 * MB> two{};
  constexpr std::integral_constant<int, N> all{};
  auto nothing = [](int) {};

  if constexpr (TWICE) {
    // All runs for hi lo and lo hi, then all of them again, 64 k at a time, for hi hi.
    // LDS is a ring of five stages of one operand: run k's are 2 k and 2 k + 1, modulo
    // 5.  While run k is multiplied, the first operand of run k + 2 goes to the stage
    // before them (everyone has read it: the last barrier), and the second, once
    // everyone has read run k, to its first stage.  Before that barrier run k + 1 has
    // landed, and only the loads of the first operand of k + 2 may be on their way.
    static_assert(MB == 4 && !SLICE && 5 * BYTES <= 163840, "a run's 64 products a wave, and all of the LDS");
    const int total = runs + doubles;
    auto load_p2 = [&](int k, uint32_t s, int i) INLINE {
      load_twice(bp, rec_p, vp[i], k, i, base + s + (uint32_t)(i * 1024));
    };
    auto load_q2 = [&](int k, uint32_t s, int i) INLINE {
      load_twice(bq, rec_q, vq[i], k, i, base + s + (uint32_t)(i * 1024));
    };
    f16x8 x0[MB], y0[MB], x1[MB], y1[MB];
    auto read = [&](uint32_t at, int b) INLINE { return *(const f16x8*)(smem + at + b * 4096); };
    auto both = [&](uint32_t p, uint32_t q, int r, f16x8 (&x)[MB], f16x8 (&y)[MB]) INLINE {
      r < MB ? (void)(x[r] = read(p, r)) : (void)(y[r - MB] = read(q, r - MB));
    };
#pragma unroll
    for (int k = 0; k < 2; k++) {
#pragma unroll
      for (int i = 0; i < N; i++) load_p2(k, (uint32_t)(2 * k * BYTES), i);
#pragma unroll
      for (int i = 0; i < N; i++) load_q2(k, (uint32_t)((2 * k + 1) * BYTES), i);
    }
    wait_loads<2 * N>();
    barrier();
    uint32_t sp = 0, sq = BYTES;  // the stages of run k
#pragma unroll
    for (int r = 0; r < 2 * MB; r++) both(at_p[0] + sp, at_q[2] + sq, r, x0, y0);
    auto run = [&](int k, auto crossc, auto firstc) INLINE {
      constexpr bool CROSS = decltype(crossc)::value;
      // Which quarter (hi of k 0-15, hi of 16-31, then lo or the next run's hi) of
      // either operand a part of 16 k takes.
      constexpr int P[4] = {0, CROSS ? 2 : 1, CROSS ? 1 : 2, 3}, Q[4] = {CROSS ? 2 : 0, CROSS ? 0 : 1, CROSS ? 3 : 2, CROSS ? 1 : 3};
      const uint32_t before = sp == 0 ? 4 * BYTES : sp - BYTES, old = sp;
      part(firstc, hi, x0, y0, two, [&](int r) { both(at_p[P[1]] + sp, at_q[Q[1]] + sq, r, x1, y1); }, all,
           [&](int i) { load_p2(k + 2, before, i); });
      part(lo, hi, x1, y1, two, [&](int r) { both(at_p[P[2]] + sp, at_q[Q[2]] + sq, r, x0, y0); }, none, nothing);
      part(lo, hi, x0, y0, two, [&](int r) { both(at_p[P[3]] + sp, at_q[Q[3]] + sq, r, x1, y1); }, none, nothing);
      wait_loads<N, 0>();
      barrier();
      sp = sp >= 3 * BYTES ? sp - 3 * BYTES : sp + 2 * BYTES;
      sq = sq >= 3 * BYTES ? sq - 3 * BYTES : sq + 2 * BYTES;
      const uint32_t next = k + 1 < runs ? at_q[2] : at_q[0];
      part(lo, hi, x1, y1, two, [&](int r) { both(at_p[0] + sp, next + sq, r, x0, y0); }, all,
           [&](int i) { load_q2(k + 2, old, i); });
    };
    run(0, std::true_type(), std::true_type());
#pragma unroll 1
    for (int k = 1; k < runs; k++) run(k, std::true_type(), std::false_type());
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
      for (int n = 0; n < MB; n++) {
        // (One block at a time: all of them find no room outside the accumulation registers.)
        asm volatile("" : "+a"(acc[m][n]));
        acc[m][n] *= a.lo_down;
        asm volatile("" : "+a"(acc[m][n]));
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll 1
    for (int k = runs; k < total; k++) run(k, std::false_type(), std::false_type());
  } else if constexpr (NS > 2) {
    // One workgroup's matrix instructions hide neither a load's nor an LDS
    // read's way: NS - 1 runs are in flight, and one is read ahead.
    auto load = [&](int k, int s) INLINE {
#pragma unroll
      for (int i = 0; i < N; i++) {
        load_p(k, s, i);
        load_q(k, s, i);
      }
    };
#pragma unroll
    for (int k = 0; k < NS - 1; k++) load(k, k);
    f16x8 p[2][4][MB], q[2][4][MB];
    auto read = [&](int s, f16x8 (&x)[4][MB], f16x8 (&y)[4][MB]) INLINE {
      const char* const st = smem + 2 * s * BYTES;
#pragma unroll
      for (int c = 0; c < 4; c++)
#pragma unroll
        for (int b = 0; b < MB; b++) {
          x[c][b] = *(const f16x8*)(st + at_p[c] + b * 4096);
          y[c][b] = *(const f16x8*)(st + BYTES + at_q[c] + b * 4096);
        }
    };
    int s = 0;  // the stage of run k
    // Run k is in registers: its products, while run k + 1 is read.
    auto run = [&](int k, const f16x8 (&x)[4][MB], const f16x8 (&y)[4][MB], f16x8 (&nx)[4][MB], f16x8 (&ny)[4][MB],
                   auto firstc) INLINE {
      // Run k + 1 has landed, those after it are on their way; and everyone has
      // read the stage of run k - 1, which run k + NS - 1 goes to.
      wait_loads<(NS - 3) * 2 * N>();
      barrier();
      const int free = s == 0 ? NS - 1 : s - 1;
      s = s == NS - 1 ? 0 : s + 1;
      const char* const st = smem + 2 * s * BYTES;
      // The order is pinned: left alone, the reads end up behind the products.
      constexpr int Q = 6 * MB * MB, R = 8 * MB, RQ = 2 * Q / 3, L = 2 * N;
#pragma unroll
      for (int i = 0; i < Q; i++) {
        const int ks = i / (Q / 2), h = i / (MB * MB) % 3, n = i / MB % MB, m = i % MB;  // hi hi, hi lo, lo hi
        multiply(firstc.value && ks == 0 && h < (APART ? 2 : 1), h == 0, m, n, x[ks + (h == 2 ? 2 : 0)][m],
                 y[ks + (h == 1 ? 2 : 0)][n]);
#pragma unroll
        for (int r = i * R / RQ; r < (i + 1) * R / RQ && r < R; r++) {
          // In the order of use.
          const int c = r / (4 * MB) + (r / (2 * MB) % 2) * 2, b = r % MB;
          if (r / MB % 2 == 0)
            nx[c][b] = *(const f16x8*)(st + at_p[c] + b * 4096);
          else
            ny[c][b] = *(const f16x8*)(st + BYTES + at_q[c] + b * 4096);
        }
#pragma unroll
        for (int l = (i - RQ) * L / (Q - RQ); i >= RQ && l < (i - RQ + 1) * L / (Q - RQ); l++)
          l < N ? load_p(k + NS - 1, free, l) : load_q(k + NS - 1, free, l - N);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    wait_loads<(NS - 2) * 2 * N>();
    barrier();
    read(0, p[0], q[0]);
    run(0, p[0], q[0], p[1], q[1], std::true_type());
#pragma unroll 1
    for (int k = 1; k < runs; k += 2) {
      run(k, p[1], q[1], p[0], q[0], std::false_type());
      if (k + 1 < runs) run(k + 1, p[0], q[0], p[1], q[1], std::false_type());
    }
  } else {
    f16x8 ph0[MB], ph1[MB], pl[MB], qh0[MB], qh1[MB], ql[MB];
    // Runs 0 .. NS - 2, and the first operand's run NS - 1.
#pragma unroll
    for (int k = 0; k < NS - 1; k++) {
#pragma unroll
      for (int i = 0; i < N; i++) load_p(k, k, i);
#pragma unroll
      for (int i = 0; i < N; i++) load_q(k, k, i);
    }
    wait_loads<(NS - 2) * 2 * N>();
    barrier();
#pragma unroll
    for (int i = 0; i < N; i++) load_p(NS - 1, NS - 1, i);
#pragma unroll
    for (int b = 0; b < MB; b++) {
      ph0[b] = read_p(0, 0, 0, b);
      qh0[b] = read_q(0, 0, 0, b);
    }
    // Run k in stage S, whose first hi fragments are in registers.  The stage
    // before it gets the second operand's run k + NS - 1; S itself, once every
    // wave has read it (and run k + 1 has landed), the first operand's run k + NS.
    auto run = [&](int k, auto sc, auto firstc) INLINE {
      constexpr int S = decltype(sc)::value, NEXT = (S + 1) % NS, LAST = (S + NS - 1) % NS;
      part(firstc, hi, ph0, qh0, two,
           [&](int r) { r < MB ? (void)(ql[r] = read_q(S, 0, 1, r)) : (void)(pl[r - MB] = read_p(S, 0, 1, r - MB)); }, all,
           [&](int i) { load_q(k + NS - 1, LAST, i); });
      part(std::integral_constant<bool, firstc.value && APART>(), lo, ph0, ql, one, [&](int r) { ph1[r] = read_p(S, 1, 0, r); }, none, nothing);
      part(std::false_type(), lo, pl, qh0, one, [&](int r) { qh1[r] = read_q(S, 1, 0, r); }, none, nothing);
      part(std::false_type(), hi, ph1, qh1, two,
           [&](int r) { r < MB ? (void)(ql[r] = read_q(S, 1, 1, r)) : (void)(pl[r - MB] = read_p(S, 1, 1, r - MB)); }, none,
           nothing);
      wait_loads<(NS - 2) * 2 * N, 0>();
      barrier();
      part(std::false_type(), lo, ph1, ql, one, [&](int r) { ph0[r] = read_p(NEXT, 0, 0, r); }, all,
           [&](int i) { load_p(k + NS, S, i); });
      part(std::false_type(), lo, pl, qh1, one, [&](int r) { qh0[r] = read_q(NEXT, 0, 0, r); }, none, nothing);
    };
    run(0, std::integral_constant<int, 0>(), std::true_type());
#pragma unroll 1
    for (int k = 1; k < runs; k += NS) {
      run(k, std::integral_constant<int, 1>(), std::false_type());
      if (k + NS - 1 < runs) run(k + NS - 1, std::integral_constant<int, 0>(), std::false_type());
    }
  }
  // The last loads (zeros) have landed, and everyone has read the stages.
  wait_all();
  barrier();

  // A lane of block (m, n): C column lane % 32, rows 8 q + 4 (lane / 32) + 0..3.
  // Blocks are staged one column (MB of them) at a time, rows of PITCH words.
  constexpr int PITCH = 36;
  char* const stage = smem + wave * (MB * 32 * PITCH * 4);
  char* const st = stage;
  const int r = lane & 31, upper = lane >> 5;
  const int m0 = T * mt + 32 * MB * wm, n0 = T * nt + 32 * MB * wn;
#pragma unroll
  for (int n = 0; n < MB; n++) {
#pragma unroll
    for (int m = 0; m < MB; m++) {
      if constexpr (MB == 4) asm volatile("" : "+a"(acc[m][n]));
      const int row0 = m0 + 32 * m, col = n0 + 32 * n + r;
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; j++) v[j] = (APART ? __builtin_fmaf(low[APART ? m : 0][APART ? n : 0][j], a.lo_down, acc[m][n][j]) : acc[m][n][j]) * a.mul;
      // (A power of two and the scale apart: together they may be below f32's normal
      // numbers where the result is not.)
      if constexpr (STAGE == ORTHO_LAST) {
#pragma unroll
        for (int j = 0; j < 16; j++) v[j] *= a.scale;
      }
      if constexpr (STAGE == ORTHO_POLY) {
        u32x2 (&o)[8] = own[EARLY ? n * MB + m : 0];
        if constexpr (!EARLY) fetch(m, n, o);
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const u32x2 x = o[q], y = o[4 + q];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const float w =
                __builtin_fmaf(half_value(y[j >> 1] >> (16 * (j & 1))), a.lo_down, half_value(x[j >> 1] >> (16 * (j & 1))));
            v[4 * q + j] = __builtin_fmaf(a.p_mul, w, v[4 * q + j]);
            if (row0 + 8 * q + 4 * upper + j == col) v[4 * q + j] += a.diag;
          }
        }
      }
      if constexpr (SLICE) {
        float* const o = a.sums + (int64_t)block * (T * T) + (32 * MB * wn + 32 * n + r) * T + 32 * MB * wm + 32 * m;
#pragma unroll
        for (int q = 0; q < 4; q++)
          *(f32x4*)(o + 8 * q + 4 * upper) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      } else if constexpr (STAGE == ORTHO_LAST) {
        // A row of the output at a time, four elements a lane: 32 x 32 in f32, chunk
        // c of row i at c ^ (i % 8).
        float* const f = (float*)st;
        if (a.flip) {
#pragma unroll
          for (int q = 0; q < 4; q++)
            *(f32x4*)(st + r * 128 + (((2 * q + upper) ^ (r & 7)) << 4)) =
                f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        } else {
#pragma unroll
          for (int j = 0; j < 16; j++) {
            const int i = 8 * (j >> 2) + 4 * upper + (j & 3);
            f[32 * i + (((r >> 2) ^ (i & 7)) << 2) + (r & 3)] = v[j];
          }
        }
        asm volatile("" ::: "memory");  // a wave's LDS accesses run in order
        const int out0 = a.flip ? n0 + 32 * n : row0, in0 = a.flip ? row0 : n0 + 32 * n;
        const int outs = a.flip ? a.cols : a.rows, ins = a.flip ? a.rows : a.cols;
#pragma unroll
        for (int it = 0; it < 4; it++) {
          const int i = 8 * it + (lane >> 3), c = lane & 7;
          const f32x4 w = *(const f32x4*)(st + i * 128 + ((c ^ (i & 7)) << 4));
          const int left = out0 + i < outs ? ins - in0 - 4 * c : 0;
          const int64_t o = mat * a.out_mat + (int64_t)(out0 + i) * a.out_row + in0 + 4 * c;
          if (a.out_dtype == CBD_F32) {
            float* const d = (float*)a.out + o;
            if (left >= 4) {
              *(f32x4u*)d = w;
            } else {
#pragma unroll
              for (int j = 0; j < 3; j++)
                if (j < left) d[j] = w[j];
            }
          } else {
            uint16_t* const d = (uint16_t*)a.out + o;
            const u32x2 b = {dev::bf16_pack2(w[0], w[1]), dev::bf16_pack2(w[2], w[3])};
            if (left >= 4) {
              *(u32x2u*)d = b;
            } else {
#pragma unroll
              for (int j = 0; j < 3; j++)
                if (j < left) d[j] = (uint16_t)(b[j >> 1] >> (16 * (j & 1)));
            }
          }
        }
        asm volatile("" ::: "memory");
      } else {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; j++) {
          const int row = row0 + 8 * (j >> 2) + 4 * upper + (j & 3);
          w[j] = row < a.rows && col < a.cols ? split(v[j], a.lo_up) : 0u;
        }
        // As C^T, row `col`: four neighbouring elements of a lane at a time, both
        // halves of one in a word.
        uint32_t* const t = (uint32_t*)(stage + m * (32 * PITCH * 4));
#pragma unroll
        for (int q = 0; q < 4; q++)
          *(u32x4*)(t + PITCH * r + 8 * q + 4 * upper) = u32x4{w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (STAGE != ORTHO_LAST && !SLICE) {
      // A column of blocks leaves: eight elements a lane, their hi and their lo.
      asm volatile("" ::: "memory");  // a wave's LDS accesses run in order
      auto leave = [&](const uint32_t (&w)[8], uint16_t* o) INLINE {
        u32x4 hi, lo;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          hi[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x05040100u);
          lo[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x07060302u);
        }
        *(u32x4*)o = hi;
        *(u32x4*)(o + 32) = lo;
      };
#pragma unroll
      for (int m = 0; m < MB; m++)
#pragma unroll
        for (int it = 0; it < 2; it++) {
          const int i = 16 * it + (lane >> 2), e = 8 * (lane & 3);
          const uint32_t* const t = (const uint32_t*)(stage + m * (32 * PITCH * 4));
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 2; j++) {
            const u32x4 x = *(const u32x4*)(t + PITCH * i + e + 4 * j);
#pragma unroll
            for (int k = 0; k < 4; k++) w[4 * j + k] = x[k];
          }
          leave(w, a.ct + mat * a.ct_mat + (int64_t)(n0 + 32 * n + i) * a.ldct + ((m0 >> 5) + m) * 64 + e);
          // A diagonal tile of a symmetric matrix has both directions already.
          if (!SYM || mt != nt) {
#pragma unroll
            for (int k = 0; k < 8; k++) w[k] = t[PITCH * (e + k) + i];
            leave(w, a.c + mat * a.c_mat + (int64_t)(m0 + 32 * m + i) * a.ldc + ((n0 >> 5) + n) * 64 + e);
          }
        }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// A block of 32 x 32 of A: its slices' sums, added in their order, in both directions.
__global__ __launch_bounds__(THREADS) void ortho_join_kernel(const OrthoArgs a) {
  __shared__ uint32_t block[32][33];
  const int t = blockIdx.x >> 2, per = a.tiles_n * (a.tiles_n + 1) / 2, mat = t / per;
  const int hm = blockIdx.x & 1, hn = blockIdx.x >> 1 & 1, i = threadIdx.x >> 3, e = 4 * (threadIdx.x & 7);
  int mt, nt;
  upper_tile(t - mat * per, a.tiles_n, 4, mt, nt);
  const float* const p = a.sums + (int64_t)t * a.slices * 4096 + (32 * hn + i) * 64 + 32 * hm + e;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = 0; s < a.slices; s++) v += *(const f32x4*)(p + (int64_t)s * 4096);
  const int row0 = 64 * mt + 32 * hm, col0 = 64 * nt + 32 * hn;
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    w[j] = row0 + e + j < a.rows && col0 + i < a.cols ? split(v[j] * a.mul, a.lo_up) : 0u;
    block[i][e + j] = w[j];
  }
  auto leave = [&](uint16_t* o) INLINE {
    *(u32x2*)o = u32x2{__builtin_amdgcn_perm(w[1], w[0], 0x05040100u), __builtin_amdgcn_perm(w[3], w[2], 0x05040100u)};
    *(u32x2*)(o + 32) =
        u32x2{__builtin_amdgcn_perm(w[1], w[0], 0x07060302u), __builtin_amdgcn_perm(w[3], w[2], 0x07060302u)};
  };
  leave(a.ct + mat * a.ct_mat + (int64_t)(col0 + i) * a.ldct + (row0 >> 5) * 64 + e);
  if (mt == nt) return;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; j++) w[j] = block[e + j][i];
  leave(a.c + mat * a.c_mat + (int64_t)(row0 + i) * a.ldc + (col0 >> 5) * 64 + e);
}

// ---- the input: norm, then both directions as two halves a value

template <typename T>
__device__ inline float value(const void* p, int64_t i) {
  if constexpr (sizeof(T) == 4)
    return ((const float*)p)[i];
  else
    return dev::bf16_to_f32(((const uint16_t*)p)[i]);
}

// Sums of squares in 64 bits: wave i of a matrix's takes rows i, i + all, ...,
// 16 bytes a lane at any alignment.
template <typename T>
__global__ __launch_bounds__(THREADS) void ortho_norm_kernel(const OrthoSplit a) {
  constexpr int V = 16 / sizeof(T), WAVES = THREADS / 64;
  typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
  typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
  using any = std::conditional_t<sizeof(T) == 4, u32x4_4, u32x4_2>;
  __shared__ double part[WAVES];
  const int64_t mat = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double s[2] = {0.0, 0.0};
  auto add = [&](int j, float f) INLINE { s[j & 1] = __builtin_fma((double)f, (double)f, s[j & 1]); };
  for (int64_t row = blockIdx.x * WAVES + wave; row < a.rows; row += kOrthoParts * WAVES) {
    const T* const p = (const T*)a.in + mat * a.in_mat + row * a.in_row;
    int col = V * lane;
#pragma unroll 4
    for (; col + V <= a.cols; col += 64 * V) {
      const u32x4 v = *(const any*)(p + col);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if constexpr (sizeof(T) == 4) {
          add(j, __uint_as_float(v[j]));
        } else {
          add(0, __uint_as_float(v[j] << 16));
          add(1, __uint_as_float(v[j] & 0xffff0000u));
        }
      }
    }
    for (int j = 0; j < V && col + j < a.cols; j++) add(j, value<T>(p, col + j));
  }
  double sum = s[0] + s[1];
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m, 64);
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.partial[mat * kOrthoParts + blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// 64 x 64 elements of a matrix.
template <typename T>
__global__ __launch_bounds__(THREADS) void ortho_split_kernel(const OrthoSplit a) {
  __shared__ uint32_t tile[64][65];
  const int64_t mat = blockIdx.z;
  const int row0 = blockIdx.y * 64, col0 = blockIdx.x * 64, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // (From inside always: loads in branches would each be waited for.)
  const int col = col0 + lane < a.cols ? col0 + lane : a.cols - 1;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int row = row0 + 4 * i + wave < a.rows ? row0 + 4 * i + wave : a.rows - 1;
    v[i] = value<T>(a.in, mat * a.in_mat + (int64_t)row * a.in_row + col);
  }
#pragma unroll
  for (int i = 0; i < 16; i++)
    if (row0 + 4 * i + wave >= a.rows || col0 + lane >= a.cols) v[i] = 0.f;
  // Every wave adds the parts in the same order.
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kOrthoParts / 64; i++) s += a.partial[mat * kOrthoParts + 64 * i + lane];
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m, 64);
  // The factor as m 2^e: it may be past f32, and products in 64 bits take a third
  // of the time that 16 x 256 x 512 take (14 us; 9 so).
  int e2;
  float m2 = (float)frexp(a.up / (__builtin_sqrt(s) + a.eps), &e2);
  if (s == 0.0) m2 = 0.f;  // zeros, also where the inverse of eps is past f64
#pragma unroll
  for (int i = 0; i < 16; i++) tile[4 * i + wave][lane] = split(ldexpf(v[i], e2) * m2, a.lo_up);
  __syncthreads();
  // A row of the tile is two runs, 16 pieces of 16 bytes: a lane takes one.
  const int piece = lane & 15, e = 32 * (piece >> 3) + 8 * (piece & 3);
  const uint32_t sel = piece & 4 ? 0x07060302u : 0x05040100u;  // of two values, both lo or both hi
  uint16_t* const x = a.x + mat * a.x_mat + (int64_t)row0 * a.ldx + col0 * 2 + 8 * piece;
  uint16_t* const xt = a.xt + mat * a.xt_mat + (int64_t)col0 * a.ldxt + row0 * 2 + 8 * piece;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int row = 16 * i + 4 * wave + (lane >> 4);
    u32x4 u, v;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      u[j] = __builtin_amdgcn_perm(tile[row][e + 2 * j + 1], tile[row][e + 2 * j], sel);
      v[j] = __builtin_amdgcn_perm(tile[e + 2 * j + 1][row], tile[e + 2 * j][row], sel);
    }
    // Past the caches: 8 matrices of 4096 x 2048 in bf16 103 us, otherwise 113, in f32
    // 124 / 134; 16 of 256 x 512 alike.
    __builtin_nontemporal_store(u, (u32x4*)(x + (int64_t)row * a.ldx));
    __builtin_nontemporal_store(v, (u32x4*)(xt + (int64_t)row * a.ldxt));
  }
}

template <int STAGE>
const void* pick(int tile, int64_t tiles, bool twice) {
  if (tile == 256)
    return twice ? (const void*)&ortho_product_kernel<4, STAGE, 2, true> : (const void*)&ortho_product_kernel<4, STAGE, 2>;
  if (tile == 64) return (const void*)&ortho_product_kernel<1, STAGE, 5>;
  return tiles <= 256 ? (const void*)&ortho_product_kernel<2, STAGE, 4>
                      : (const void*)&ortho_product_kernel<2, STAGE, 2>;
}

}  // namespace

int launch_ortho_norm(const OrthoSplit& a, int64_t matrices, void* stream) {
  void* args[] = {const_cast<OrthoSplit*>(&a)};
  const void* k = a.dtype == CBD_F32 ? (const void*)&ortho_norm_kernel<float> : (const void*)&ortho_norm_kernel<uint16_t>;
  return (int)hipLaunchKernel(k, dim3(kOrthoParts, (unsigned)matrices), dim3(THREADS), args, 0, (hipStream_t)stream);
}
int launch_ortho_split(const OrthoSplit& a, int64_t matrices, void* stream) {
  void* args[] = {const_cast<OrthoSplit*>(&a)};
  const void* k =
      a.dtype == CBD_F32 ? (const void*)&ortho_split_kernel<float> : (const void*)&ortho_split_kernel<uint16_t>;
  return (int)hipLaunchKernel(k, dim3((unsigned)((a.cols + 63) / 64), (unsigned)((a.rows + 63) / 64), (unsigned)matrices),
                              dim3(THREADS), args, 0, (hipStream_t)stream);
}
int launch_ortho_join(const OrthoArgs& a, int64_t matrices, void* stream) {
  void* args[] = {const_cast<OrthoArgs*>(&a)};
  const int64_t tiles = (int64_t)a.tiles_n * (a.tiles_n + 1) / 2 * matrices;
  return (int)hipLaunchKernel((const void*)&ortho_join_kernel, dim3((unsigned)(4 * tiles)), dim3(THREADS), args, 0,
                              (hipStream_t)stream);
}
int launch_ortho_product(const OrthoArgs& a, int stage, int tile, int64_t matrices, void* stream) {
  void* args[] = {const_cast<OrthoArgs*>(&a)};
  const bool sym = stage == ORTHO_SQUARE || stage == ORTHO_POLY || stage == ORTHO_SLICE;
  const int64_t per = stage == ORTHO_SLICE ? (int64_t)a.tiles_m * (a.tiles_m + 1) / 2 * a.slices
                      : sym                ? (int64_t)a.tiles_m * (a.tiles_m + 1) / 2 : (int64_t)a.tiles_m * a.tiles_n;
  const void* k = stage == ORTHO_SLICE ? (const void*)&ortho_product_kernel<1, ORTHO_SLICE, 5>
                  : stage == ORTHO_SQUARE ? pick<ORTHO_SQUARE>(tile, per * matrices, a.lo_up != 1.f)
                  : stage == ORTHO_POLY ? pick<ORTHO_POLY>(tile, per * matrices, a.lo_up != 1.f)
                  : stage == ORTHO_STEP ? pick<ORTHO_STEP>(tile, per * matrices, a.lo_up != 1.f)
                                        : pick<ORTHO_LAST>(tile, per * matrices, a.lo_up != 1.f);
  return (int)hipLaunchKernel(k, dim3((unsigned)(per * matrices)), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
