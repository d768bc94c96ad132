// kern_expert_stream.hip -- bf16 expert products with few rows an expert
// (served tokens), on v_mfma_f32_16x16x32_bf16: the weights stream once from
// HBM through registers, without LDS.
//
// A workgroup of 4 waves computes a slice of features by up to 32 rows of one
// expert; the waves take turns in the contracted steps and their sums are
// joined through LDS at the end, in a fixed order.  Each wave keeps DEPTH
// steps' loads in flight; steps past the end load zeros (out of the buffer's
// range), so the loop has no branch.
//
//   AK (weight rows k-contiguous): 32 features, steps of 64 k.  A lane loads
//     16 bytes of one feature's row: 8 consecutive k, as the MFMA wants them.
//   AM (features contiguous): 128 features, steps of 32 k.  A lane loads 16
//     bytes (8 features) of each of 8 consecutive k; v_perm pairs neighbouring
//     k rows into the k vectors of 8 MFMAs, the j-th of which has feature
//     8 i + j as its row i, so a lane ends with 8 neighbouring features.
//
// Rows of the activations are read straight from L2 (every workgroup of an
// expert reads the same few).  Any alignment of 2 bytes will do.
//
// Bound: HBM, one pass over the weights of the experts that have rows.  64
// experts of 2048 x 1408 with 8 rows each: AK 73 us (5.1 TB/s), AM 66 us (5.6);
// 8 of them with a row each 12.5 us, where the way to the first load (row
// ranges, tile, addresses) counts.  AK has one step in flight a wave and 8
// waves a SIMD: with two and 5 waves 77 us, four and 3 waves 80, seven and 2
// waves 103; non-temporal loads 87.
#include <type_traits>

#include "cbd_device.h"
#include "expert_device.h"

namespace cbd {
namespace {

typedef short bf16x8 __attribute__((__vector_size__(8 * sizeof(short))));
typedef float f32x4 __attribute__((__vector_size__(4 * sizeof(float))));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));

constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;
constexpr int BN = 32;

// Elements [0, n) of p (n < 8), zeros after them.
__device__ inline u32x4 part8(const uint16_t* p, int n) {
  u32x4 x = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 7; j++)
    if (j < n) x[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
  return x;
}

// Values [lo, n) of 8 of a row, rounded once.
__device__ inline void store8(uint16_t* o, const float* v, int lo, int n) {
  if (lo <= 0 && n >= 8) {
    *(u32x4u*)o = u32x4{dev::bf16_pack2(v[0], v[1]), dev::bf16_pack2(v[2], v[3]), dev::bf16_pack2(v[4], v[5]),
                        dev::bf16_pack2(v[6], v[7])};
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (j >= lo && j < n) o[j] = (uint16_t)dev::bf16_rne(v[j]);
  }
}

template <int FORM>
struct Shape {
  static constexpr bool AK = FORM == EXPERT_AK;
  static constexpr int BM = AK ? 32 : 128;
  static constexpr int BK = AK ? 64 : 32;
  static constexpr int WL = AK ? 4 : 8;         // weight loads of a step
  static constexpr int BLOCKS = AK ? 2 : 8;     // 16-feature blocks
};

template <int FORM>
__global__ __launch_bounds__(THREADS, FORM == EXPERT_AK ? 8 : 2) void expert_stream_kernel(const ExpertArgs a) {
  using S = Shape<FORM>;
  constexpr bool AK = S::AK;
  // Sums of the waves (AM: of 16 rows at a time).
  __shared__ __attribute__((aligned(16))) f32x4 sums[WAVES][AK ? 4 : 8][64];
  dev::RowTiles tiles;
  tiles.init(a, BN);
  const dev::ExpertTile t = tiles.at(a, blockIdx.x, BN);
  if (!t.ok) return;
  const int lane = threadIdx.x & 63, wave = dev::uniform((int)(threadIdx.x >> 6));
  const int g = lane >> 4, i16 = lane & 15;
  const int K = t.e < a.E ? a.K : 0;  // rows past the last expert's: zeros
  const int n0 = t.begin;
  const int nrows = t.end - n0;
  // AM: the last slice starts earlier, so that no 16 bytes pass the row's end.
  const dev::FeatureSlice slice =
      AK ? dev::FeatureSlice{t.m_tile * S::BM, 0} : dev::feature_slice(t.m_tile, S::BM, a.M);
  const int m0 = slice.m0;
  const uint16_t* const w =
      (const uint16_t*)a.a + (t.e < a.E ? t.e * a.a_expert : 0) + (AK ? m0 * a.lda : (int64_t)m0);
  const uint16_t* const x = (const uint16_t*)a.b + n0 * a.ldb;
  const uint32_t ld = (uint32_t)a.lda * 2u;
  const int mrows = a.M - m0;
  // AM with fewer than 128 features: the weights are loaded by elements where
  // a 16-byte chunk would pass the row's end.
  const bool narrow = !AK && a.M < S::BM;

  auto work = [&](auto nbc) CBD_INLINE {
    constexpr int NB = decltype(nbc)::value;
    constexpr int XL = (AK ? 2 : 1) * NB;          // activation loads of a step
    constexpr int DEPTH = AK ? 1 : 2;
    f32x4 acc[S::BLOCKS][NB];
#pragma unroll
    for (int m = 0; m < S::BLOCKS; m++)
#pragma unroll
      for (int n = 0; n < NB; n++) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};

    const auto rw = dev::rsrc(w, K > 0 ? (uint32_t)(AK ? ((int64_t)((mrows < S::BM ? mrows : S::BM) - 1) * a.lda + K) * 2
                                                       : ((int64_t)(K - 1) * a.lda + mrows) * 2)
                                       : 0u);
    const auto rx = dev::rsrc(x, K > 0 ? (uint32_t)(((int64_t)(nrows - 1) * a.ldb + K) * 2) : 0u);
    uint32_t wo[S::WL], xo[NB];
    if constexpr (AK) {
#pragma unroll
      for (int m = 0; m < 2; m++) {
        const int r = 16 * m + i16 < mrows ? 16 * m + i16 : mrows - 1;  // past the edge: any row
        wo[2 * m] = (uint32_t)r * ld + (uint32_t)g * 16u;
        wo[2 * m + 1] = wo[2 * m] + 64u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) wo[i] = (uint32_t)(8 * g + i) * ld + (uint32_t)i16 * 16u;
    }
#pragma unroll
    for (int n = 0; n < NB; n++) {
      const int r = 16 * n + i16 < nrows ? 16 * n + i16 : nrows - 1;
      xo[n] = (uint32_t)r * ((uint32_t)a.ldb * 2u) + (uint32_t)g * 16u;
    }
    const int steps = (K + S::BK - 1) / S::BK;
    u32x4 wv[DEPTH][S::WL], xv[DEPTH][XL];
    auto load = [&](int d, int s) CBD_INLINE {
      const int k = s * S::BK + 8 * g;
      // Whole chunks of 8 k only; what is left of K is added at the end.
      const bool in0 = k + 8 <= K, in1 = AK && k + 40 <= K;
      if constexpr (AK) {
        const uint32_t so = (uint32_t)s * 128u;
#pragma unroll
        for (int m = 0; m < 2; m++) {
          wv[d][2 * m] = __builtin_amdgcn_raw_buffer_load_b128(rw, in0 ? wo[2 * m] + so : dev::kOOB, 0, 0);
          wv[d][2 * m + 1] = __builtin_amdgcn_raw_buffer_load_b128(rw, in1 ? wo[2 * m + 1] + so : dev::kOOB, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NB; n++) {
          xv[d][2 * n] = __builtin_amdgcn_raw_buffer_load_b128(rx, in0 ? xo[n] + so : dev::kOOB, 0, 0);
          xv[d][2 * n + 1] = __builtin_amdgcn_raw_buffer_load_b128(rx, in1 ? xo[n] + so + 64u : dev::kOOB, 0, 0);
        }
      } else {
        const uint32_t so = (uint32_t)s * (32u * ld);
#pragma unroll
        for (int i = 0; i < 8; i++)
          wv[d][i] = __builtin_amdgcn_raw_buffer_load_b128(rw, in0 ? wo[i] + so : dev::kOOB, 0, 0);
#pragma unroll
        for (int n = 0; n < NB; n++)
          xv[d][n] = __builtin_amdgcn_raw_buffer_load_b128(rx, in0 ? xo[n] + (uint32_t)s * 64u : dev::kOOB, 0, 0);
      }
    };
    // The products of one step's registers.
    auto multiply = [&](const u32x4 (&wr)[S::WL], const u32x4 (&xr)[XL]) CBD_INLINE {
      if constexpr (AK) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int m = 0; m < 2; m++)
#pragma unroll
            for (int n = 0; n < NB; n++)
              acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wr[2 * m + h]),
                                                                  __builtin_bit_cast(bf16x8, xr[2 * n + h]),
                                                                  acc[m][n], 0, 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          u32x4 v;  // k vector of feature 8 i16 + j
#pragma unroll
          for (int p = 0; p < 4; p++)
            v[p] = __builtin_amdgcn_perm(wr[2 * p + 1][j >> 1], wr[2 * p][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int n = 0; n < NB; n++)
            acc[j][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v),
                                                                __builtin_bit_cast(bf16x8, xr[n]), acc[j][n], 0, 0, 0);
        }
      }
    };
    if (!narrow) {
#pragma unroll
      for (int d = 0; d < DEPTH; d++) load(d, wave + WAVES * d);
#pragma unroll 1
      for (int s = wave; s < steps; s += WAVES * DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
          multiply(wv[d], xv[d]);
          load(d, s + WAVES * (d + DEPTH));
        }
      }
    }
    // The last K % 8 (narrow: all k, 8 at a time), by elements, on lanes 0..15.
    if (wave == 0) {
#pragma unroll 1
      for (int k = narrow ? 0 : K & ~7; k < K; k += 8) {
        const int left = K - k;
        u32x4 wt[S::WL], xt[XL];
#pragma unroll
        for (int i = 0; i < S::WL; i++) wt[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < XL; i++) xt[i] = u32x4{0u, 0u, 0u, 0u};
        if (g == 0) {
          if constexpr (AK) {
#pragma unroll
            for (int m = 0; m < 2; m++) {
              const int r = 16 * m + i16 < mrows ? 16 * m + i16 : mrows - 1;
              wt[2 * m] = part8(w + r * a.lda + k, left);
            }
          } else {
            const int f = mrows - 8 * i16;
#pragma unroll
            for (int i = 0; i < 8; i++)
              if (i < left && f > 0) {
                const uint16_t* p = w + (k + i) * a.lda + 8 * i16;
                wt[i] = f >= 8 ? (u32x4) * (const u32x4u*)p : part8(p, f);
              }
          }
#pragma unroll
          for (int n = 0; n < NB; n++) {
            const int r = 16 * n + i16 < nrows ? 16 * n + i16 : nrows - 1;
            const uint16_t* p = x + r * a.ldb + k;
            xt[AK ? 2 * n : n] = left >= 8 ? (u32x4) * (const u32x4u*)p : part8(p, left);
          }
        }
        multiply(wt, xt);
      }
    }
    // Join the waves' sums.  A lane of a block: row lane % 16, features (AM:
    // of its 16) 4 (lane / 16) + 0..3.
    uint16_t* const out = (uint16_t*)a.out + n0 * a.ldo + m0;
    if constexpr (AK) {
#pragma unroll
      for (int n = 0; n < NB; n++)
#pragma unroll
        for (int m = 0; m < 2; m++) sums[wave][n * 2 + m][lane] = acc[m][n];
      __syncthreads();
      // 32 features x 32 rows: thread = 4 features of a row.
      const int n = threadIdx.x >> 7, m = (threadIdx.x >> 6) & 1, row = 16 * n + i16, f = 16 * m + 4 * g;
      if (n < NB && row < nrows) {
        f32x4 v = sums[0][n * 2 + m][lane];
#pragma unroll
        for (int q = 1; q < WAVES; q++) v += sums[q][n * 2 + m][lane];
        uint16_t* o = out + row * a.ldo + f;
        const uint32_t lo = dev::bf16_pack2(v[0], v[1]), hi = dev::bf16_pack2(v[2], v[3]);
        if (f + 3 < mrows) {
          typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
          *(u32x2u*)o = u32x2u{lo, hi};
        } else {
          if (f < mrows) o[0] = (uint16_t)lo;
          if (f + 1 < mrows) o[1] = (uint16_t)(lo >> 16);
          if (f + 2 < mrows) o[2] = (uint16_t)hi;
        }
      }
    } else {
      // Wave r of 4 takes value r of every lane: features 8 (4 g + r) + 0..7.
#pragma unroll
      for (int n = 0; n < NB; n++) {
        const int row = 16 * n + i16, f = 8 * (4 * g + wave);
        if (n > 0) __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; j++) sums[wave][j][lane] = acc[j][n];
        __syncthreads();
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
          v[j] = ((const float*)&sums[0][j][lane])[wave];
#pragma unroll
          for (int q = 1; q < WAVES; q++) v[j] += ((const float*)&sums[q][j][lane])[wave];
        }
        if (row < nrows && f + 8 > slice.skip && f < mrows)
          store8(out + row * a.ldo + f, v, slice.skip - f, mrows - f);
      }
    }
  };
  if (nrows <= 16)
    work(std::integral_constant<int, 1>());
  else
    work(std::integral_constant<int, 2>());
}

}  // namespace

int launch_expert_stream(const ExpertArgs& a, const ExpertLaunch& l, void* stream) {
  const void* k = l.form == EXPERT_AK ? (const void*)&expert_stream_kernel<EXPERT_AK>
                                      : (const void*)&expert_stream_kernel<EXPERT_AM>;
  void* args[] = {const_cast<ExpertArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
