// kern_expert_generic.hip -- expert products of any type, size, stride and
// alignment.
//
// A workgroup of 4 waves (2 x 2) computes a BM x BN tile (BM = BN = 128, or 64
// where 128 would leave compute units idle) of one expert with
// v_mfma_f32_16x16x4_f32; bf16 operands are widened while they are staged, so
// every product is exact and every sum f32.  Operand tiles of 16 k (64 x 64:
// 32 k) are loaded into registers two steps ahead, then written to one of two
// LDS buffers, so a step has one barrier.  Each thread keeps a pointer per
// vector that steps along k: addresses worked out anew took longer than the
// MFMAs.  Elements past the contracted length are staged as zeros on
// both sides; rows and features past an edge repeat others, and what they give
// is not stored.  So nothing beyond an edge (infinities and NaN included)
// takes part.
//
// k may be summed in any order as long as both operands agree: of each 16 k,
// lane group q = lane / 16 takes k = 4q + i at MFMA i.  A k-contiguous operand
// is staged [row][k + 4 pad] and one 16-byte LDS read gives a lane its four k; an
// operand whose features are contiguous is staged [k][features] and one read
// gives a lane MB neighbouring features of one k, which makes feature
// MB * i + block, instead of 16 * block + i, the row of lane i in a block.
//
// Bound: the f32 matrix rate (154 TFLOP/s reached by a large product; a 128 x
// 128 tile does 32 flops per loaded byte in f32).  8192 x 2048 x 2048, 4
// experts: 97 TFLOP/s; 3001 x 515 x 389, 7 experts: 29 us, of which 16 are
// MFMAs of the compute units that get two of the 357 tiles.
#include <type_traits>

#include "cbd_device.h"
#include "expert_device.h"

namespace cbd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));

constexpr int THREADS = 256;

// n (clamped to 0..4) elements from p, widened to f32; zeros after them.
__device__ inline f32x4 load4(const float* p, int n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (n >= 4) {
    v = *(const f32x4u*)p;
  } else {
    if (n > 0) v[0] = p[0];
    if (n > 1) v[1] = p[1];
    if (n > 2) v[2] = p[2];
  }
  return v;
}
__device__ inline f32x4 load4(const uint16_t* p, int n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (n >= 4) {
    const u16x4u u = *(const u16x4u*)p;
    for (int i = 0; i < 4; i++) v[i] = dev::bf16_to_f32(u[i]);
  } else {
    if (n > 0) v[0] = dev::bf16_to_f32(p[0]);
    if (n > 1) v[1] = dev::bf16_to_f32(p[1]);
    if (n > 2) v[2] = dev::bf16_to_f32(p[2]);
  }
  return v;
}

// Stores v[0..n) (n clamped to 0..4), rounded once.
__device__ inline void store4(float* p, f32x4 v, int n, bool add) {
  if (add) v += load4(p, n);
  if (n >= 4) {
    *(f32x4u*)p = v;
  } else {
    for (int i = 0; i < 3; i++)
      if (i < n) p[i] = v[i];
  }
}
__device__ inline void store4(uint16_t* p, f32x4 v, int n, bool add) {
  if (add) v += load4(p, n);
  u16x4u u;
  for (int i = 0; i < 4; i++) u[i] = (uint16_t)dev::bf16_rne(v[i]);
  if (n >= 4) {
    *(u16x4u*)p = u;
  } else {
    for (int i = 0; i < 3; i++)
      if (i < n) p[i] = u[i];
  }
}

// One operand of a tile: R rows (features or tokens) by BK k, R = 32 * NB.
// KC: k is contiguous in memory.
template <typename T, bool KC, int NB, int BK>
struct Operand {
  static constexpr int R = 32 * NB;
  static constexpr int ROW = KC ? BK + 4 : R + 4;     // floats per LDS row
  static constexpr int LDS = KC ? R * ROW : BK * ROW;  // floats
  static constexpr int NV = R * BK / 4 / THREADS;      // 4-vectors per thread
  static constexpr int QUADS = KC ? BK / 4 : R / 4;  // 4-vectors of a row
  const T* q[NV];  // this thread's vectors of the next step
  int64_t step;
  int feats[NV];   // feature-contiguous: features of the vector inside the operand
  int back[NV];    // and by how many it is loaded early
  bool edge;       // some of the wave's are
  f32x4 v[2][NV];  // two steps

  // p: element (row 0, k 0) of the tile; rows: inside the operand, >= 1.
  // width: features of the whole operand.
  CBD_INLINE __device__ void init(const T* p, int64_t ld, int rows, int width) {
    step = KC ? BK : BK * ld;
    const bool wide = width >= 4;
    edge = false;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int idx = i * THREADS + (int)threadIdx.x;
      const int row = idx / QUADS, col = 4 * (idx % QUADS);
      if (KC) {
        q[i] = p + (row < rows ? row : rows - 1) * ld + col;
        feats[i] = 4;
        back[i] = 0;
      } else {
        const int f = col < rows ? col : 0;
        // A vector that passes the edge is loaded from further down and moved
        // when it is staged: no wait for it in between.
        back[i] = rows - f < 4 && wide ? 4 - (rows - f) : 0;
        edge = edge || __any(back[i] != 0);
        q[i] = p + row * ld + f - back[i];
        feats[i] = rows - f + back[i];
      }
    }
  }
  // The next step, of which `left` k are inside, into registers `slot`.
  CBD_INLINE __device__ void load(int slot, int left) {
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int idx = i * THREADS + (int)threadIdx.x;
      const int k = KC ? 4 * (idx % QUADS) : idx / QUADS;
      if (left >= BK)
        v[slot][i] = KC ? load4(q[i], 4) : load4(q[i], feats[i]);
      else
        v[slot][i] = load4(q[i], KC ? left - k : k < left ? feats[i] : 0);
      q[i] += step;
    }
  }
  CBD_INLINE __device__ void stage(int slot, float* lds) const {
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int idx = i * THREADS + (int)threadIdx.x;
      f32x4 x = v[slot][i];
      if (!KC && edge) {
        if (back[i] & 1) x = f32x4{x[1], x[2], x[3], 0.f};
        if (back[i] & 2) x = f32x4{x[2], x[3], 0.f, 0.f};
      }
      *(f32x4*)(lds + (idx / QUADS) * ROW + 4 * (idx % QUADS)) = x;
    }
  }
  // Fragments of a wave's 16 * NB rows from row r0, k kb .. kb + 15:
  // f[block][i].
  CBD_INLINE __device__ static void read(const float* lds, int r0, int kb, float (&f)[NB][4]) {
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
    if (KC) {
#pragma unroll
      for (int b = 0; b < NB; b++) {
        const f32x4 x = *(const f32x4*)(lds + (r0 + 16 * b + r) * ROW + kb + 4 * q);
#pragma unroll
        for (int i = 0; i < 4; i++) f[b][i] = x[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float* s = lds + (kb + 4 * q + i) * ROW + r0 + NB * r;
#pragma unroll
        for (int b = 0; b < NB; b++) f[b][i] = s[b];
      }
    }
  }
  // Row of index i (0..15) of block b.
  __device__ static int row(int i, int b) { return KC ? 16 * b + i : NB * i + b; }
};

template <typename T, typename TO, int FORM, int NB>
__global__ __launch_bounds__(THREADS, NB == 4 ? 3 : 4) void expert_generic_kernel(const ExpertArgs a) {
  constexpr int BT = 32 * NB;
  constexpr int BK = NB == 4 ? 16 : 32;
  using OpA = Operand<T, FORM == EXPERT_AK, NB, BK>;
  using OpB = Operand<T, FORM != EXPERT_DW, NB, BK>;
  __shared__ __attribute__((aligned(16))) float lds[2][OpA::LDS + OpB::LDS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave & 1) * 16 * NB, wn = (wave >> 1) * 16 * NB;

  OpA oa;
  OpB ob;
  TO* out;
  int m0, K, mrows, nrows;
  if constexpr (FORM == EXPERT_DW) {
    dev::WeightTiles tiles;
    tiles.init(a, BT);
    const dev::ExpertTile t = tiles.at(a, blockIdx.x, BT, 0);
    K = t.end - t.begin;
    if (a.accumulate && K == 0) return;
    m0 = t.m_tile * BT;
    const int n0 = t.n_tile * BT;
    mrows = a.M - m0;
    nrows = a.N - n0;
    oa.init((const T*)a.a + (int64_t)t.begin * a.lda + m0, a.lda, mrows, a.M);
    ob.init((const T*)a.b + (int64_t)t.begin * a.ldb + n0, a.ldb, nrows, a.N);
    out = (TO*)a.out + t.e * a.o_expert + n0 * a.ldo + m0;
  } else {
    dev::RowTiles tiles;
    tiles.init(a, BT);
    const dev::ExpertTile t = tiles.at(a, blockIdx.x, BT);
    if (!t.ok) return;
    K = t.e < a.E ? a.K : 0;  // rows past the last expert's: zeros
    const int n0 = t.begin;
    m0 = t.m_tile * BT;
    mrows = a.M - m0;
    nrows = t.end - n0;
    oa.init((const T*)a.a + (t.e < a.E ? t.e * a.a_expert : 0) + (FORM == EXPERT_AK ? m0 * a.lda : (int64_t)m0),
            a.lda, mrows, a.M);
    ob.init((const T*)a.b + (int64_t)n0 * a.ldb, a.ldb, nrows, a.N);
    out = (TO*)a.out + (int64_t)n0 * a.ldo + m0;
  }
  const int live = dev::uniform((nrows - wn + 15) >> 4);  // 16-row blocks of this wave (AK, AM)
  f32x4 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; i++)
#pragma unroll
    for (int j = 0; j < NB; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto step = [&](auto sc, int k0) CBD_INLINE {
    constexpr int S = decltype(sc)::value;
    float* la = lds[S];
    float* lb = la + OpA::LDS;
    oa.stage(S, la);
    ob.stage(S, lb);
    // One barrier a step: buffer S was last read two steps ago, before the
    // previous step's barrier.
    __syncthreads();
    oa.load(S, K - k0 - 2 * BK);
    ob.load(S, K - k0 - 2 * BK);
#pragma unroll
    for (int kb = 0; kb < BK; kb += 16) {
      float fa[NB][4], fb[NB][4];
      OpA::read(la, wm, kb, fa);
      OpB::read(lb, wn, kb, fb);
#pragma unroll
      for (int y = 0; y < NB; y++) {
        // Whole 16-row blocks past the expert's rows are left out.
        if (FORM != EXPERT_DW && y >= live) break;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int x = 0; x < NB; x++)
            acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[x][i], fb[y][i], acc[x][y], 0, 0, 0);
      }
    }
  };
  oa.load(0, K);
  ob.load(0, K);
  oa.load(1, K - BK);
  ob.load(1, K - BK);
#pragma unroll 1
  for (int k0 = 0; k0 < K; k0 += 2 * BK) {
    step(std::integral_constant<int, 0>(), k0);
    if (k0 + BK < K) step(std::integral_constant<int, 1>(), k0 + BK);
  }

  // Lane: column (n) lane % 16 of a block, rows (m) 4 * (lane / 16) + r.
#pragma unroll
  for (int y = 0; y < NB; y++) {
    const int n = wn + OpB::row(lane & 15, y);
    if (n >= nrows) continue;
    TO* o = out + n * a.ldo;
    if constexpr (FORM == EXPERT_AK) {
#pragma unroll
      for (int x = 0; x < NB; x++) {
        const int m = wm + 16 * x + 4 * (lane >> 4);
        store4(o + m, acc[x][y], mrows - m, a.accumulate);
      }
    } else {
      // Features NB * (4q + r) + x: 4 * NB consecutive ones of a lane.
      float v[4 * NB];
#pragma unroll
      for (int x = 0; x < NB; x++)
#pragma unroll
        for (int r = 0; r < 4; r++) v[NB * r + x] = acc[x][y][r];
#pragma unroll
      for (int c = 0; c < NB; c++) {
        const int m = wm + NB * 4 * (lane >> 4) + 4 * c;
        store4(o + m, f32x4{v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]}, mrows - m, a.accumulate);
      }
    }
  }
}

template <typename T, typename TO, int FORM>
const void* pick(int bm) {
  return bm == 128 ? (const void*)&expert_generic_kernel<T, TO, FORM, 4>
                   : (const void*)&expert_generic_kernel<T, TO, FORM, 2>;
}

}  // namespace

int launch_expert_generic(const ExpertArgs& a, const ExpertLaunch& l, void* stream) {
  const void* k;
  if (l.form == EXPERT_DW)
    k = l.dtype == CBD_F32        ? pick<float, float, EXPERT_DW>(l.bm)
        : l.out_dtype == CBD_F32  ? pick<uint16_t, float, EXPERT_DW>(l.bm)
                                  : pick<uint16_t, uint16_t, EXPERT_DW>(l.bm);
  else if (l.form == EXPERT_AK)
    k = l.dtype == CBD_F32 ? pick<float, float, EXPERT_AK>(l.bm) : pick<uint16_t, uint16_t, EXPERT_AK>(l.bm);
  else
    k = l.dtype == CBD_F32 ? pick<float, float, EXPERT_AM>(l.bm) : pick<uint16_t, uint16_t, EXPERT_AM>(l.bm);
  void* args[] = {const_cast<ExpertArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
