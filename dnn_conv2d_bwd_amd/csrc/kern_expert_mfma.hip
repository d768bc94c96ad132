// kern_expert_mfma.hip -- bf16 expert products with many rows, on
// v_mfma_f32_32x32x16_bf16.
//
// A workgroup of 4 waves computes 256 features (m, the contiguous side of the
// output) x 32 * NB rows (n) of one expert in steps of 32 k; wave w owns
// features 64 w .. 64 w + 63 of all rows, so a tile that the expert's rows do
// not fill costs matrix time only for the 32-row blocks it has (rounded up to
// an even number), the same for every wave, and a wave's results leave through
// a staging buffer of its own without a barrier.
//
// Operand tiles go into a ring of NS LDS stages.  DMA: buffer_load ... lds,
// 16 bytes a lane, NS - 1 steps ahead, one barrier a step; the reads of the
// next 16 k and the loads are spread between the MFMAs.  Without DMA (rows off
// 16-byte alignment, or a contracted length that is no multiple of 8 where k
// is contiguous): through registers, one step ahead.  Lanes past an edge fetch
// zeros on both operands, so nothing beyond the rows of an expert or the
// contracted length takes part.
//
// A k-contiguous operand is staged [row][32 k], chunk c (16 bytes) of row r at
// c ^ (r / 4 % 4), and read with ds_read_b128.  A feature-contiguous one is
// staged [k][features] and read with ds_read_b64_tr_b16, which hands lane j of
// 16 the four k of feature j; its chunks are moved by 64 bytes a row so that
// the four k rows of a read sit in different banks.
#include <type_traits>

#include "expert_device.h"

namespace cbd {
namespace {

typedef short bf16x8 __attribute__((__vector_size__(8 * sizeof(short))));
typedef short bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((__vector_size__(16 * sizeof(float))));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

constexpr int BM = 256;
constexpr int BK = 32;
constexpr int THREADS = 256;

// s_waitcnt immediate: vmcnt <= n, lgkmcnt 0 (gfx9 encoding).
constexpr int waitcnt_vm_lgkm0(int n) { return (n & 15) | (7 << 4) | ((n >> 4) << 14); }

// One operand: F features (or rows) by 32 k a stage.
template <bool KC, int F, bool DMA>
struct Feed {
  static constexpr int BYTES = F * BK * 2;
  static constexpr int N = BYTES / 4096;  // 1 KiB blocks a wave fills
  static constexpr int CHUNKS = F / 8;    // 16-byte chunks of a k row (feature-contiguous)

  __device__ static int swz(int row) {
    if (KC) return (row >> 2) & 3;
    return F == 64 ? 4 * ((row >> 1) & 1) : 4 * (row & 3);
  }
  // Row (KC: of features; else of k) and chunk that a lane fills of block i.
  __device__ static int fill_row(int i) {
    const int lane = threadIdx.x & 63, j = N * (int)(threadIdx.x >> 6) + i;
    return KC ? 16 * j + (lane >> 2) : (64 / CHUNKS) * j + lane / CHUNKS;
  }
  __device__ static int fill_chunk(int i) {
    const int lane = threadIdx.x & 63;
    return (KC ? lane & 3 : lane % CHUNKS) ^ swz(fill_row(i));
  }

  const uint16_t* p;  // element (row 0, k 0)
  int64_t ld;
  int rows, K;        // features inside the operand; contracted length
  // DMA
  uint32_t voff[N];
  uint32_t soff, rec, step;
  int64_t left;       // feature-contiguous: bytes from the next step's first k row to the end
  uint64_t base;
  // registers
  u32x4 v[N];

  __device__ void init(const uint16_t* p_, int64_t ld_, int rows_, int K_) {
    p = p_;
    ld = ld_;
    rows = rows_;
    K = K_;
    if constexpr (DMA) {
      base = (uint64_t)p;
      soff = 0;
      step = (uint32_t)(BK * ld * 2);
      left = K > 0 ? ((int64_t)(K - 1) * ld + rows) * 2 : 0;
#pragma unroll
      for (int i = 0; i < N; i++) {
        const int r = fill_row(i), c = fill_chunk(i);
        voff[i] = (KC ? r < rows : 8 * c < rows) ? (uint32_t)r * (uint32_t)ld * 2u + (uint32_t)c * 16u : dev::kOOB;
      }
      if constexpr (KC) {
        rec = K > 0 ? (uint32_t)(((int64_t)((rows < F ? rows : F) - 1) * ld + K) * 2) : 0u;
        mask_tail(0);
      } else {
        clamp();
      }
    }
  }
  // Step t is the last and part of its 32 k are past the end.
  __device__ void mask_tail(int t) {
    const int over = K - t * BK;
    if (over < BK) {
#pragma unroll
      for (int i = 0; i < N; i++)
        if (8 * fill_chunk(i) >= over) voff[i] = dev::kOOB;
    }
  }
  __device__ void clamp() {
    const int64_t l = (left + 3) & ~(int64_t)3;
    rec = left <= 0 ? 0u : l > 0x7ffffffc ? 0x7ffffffcu : (uint32_t)l;
  }
  // To step t (of steps); past the last the record count is 0.
  __device__ void advance(int t, int steps) {
    if constexpr (KC) {
      soff += BK * 2;
      if (t == steps - 1) mask_tail(t);
      if (t >= steps) rec = 0;
    } else {
      base += step;
      left -= step;
      clamp();
    }
  }
  __device__ void issue(int i, uint32_t m0v) const {
    const i32x4 d = {(int)__builtin_amdgcn_readfirstlane((uint32_t)base),
                     (int)__builtin_amdgcn_readfirstlane((uint32_t)(base >> 32) & 0xffffu),
                     (int)__builtin_amdgcn_readfirstlane(rec), 0x00020000};
    const uint32_t so = __builtin_amdgcn_readfirstlane(KC ? soff : 0u);
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds\n\ts_nop 0"
                 ::"s"(m0v), "v"(voff[i]), "s"(d), "s"(so) : "memory", "m0");
#pragma clang diagnostic pop
  }

  // Through registers: step t, zeros past the edges.
  __device__ void load(int t) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int r = fill_row(i), c = fill_chunk(i);
      const int row = KC ? r : t * BK + r, col = KC ? t * BK + 8 * c : 8 * c;
      const int n = row < (KC ? rows : K) ? (KC ? K : rows) - col : 0;
      const uint16_t* s = p + row * ld + col;
      u32x4 x = {0u, 0u, 0u, 0u};
      if (n >= 8) {
        x = *(const u32x4u*)s;
      } else if (n > 0) {
#pragma unroll
        for (int j = 0; j < 7; j++)
          if (j < n) x[j >> 1] |= (uint32_t)s[j] << (16 * (j & 1));
      }
      v[i] = x;
    }
  }
  __device__ void stage(char* lds) const {
#pragma unroll
    for (int i = 0; i < N; i++)
      *(u32x4*)(lds + (N * (int)(threadIdx.x >> 6) + i) * 1024 + (threadIdx.x & 63) * 16) = v[i];
  }

  // ---- fragments: of 32 rows (block b from feature f0), 16 k (step ks).
  static constexpr int READS = KC ? 1 : 2;  // LDS reads a fragment takes
  static constexpr int REGS = KC ? 2 : F >= 128 ? 4 : 2;
  int at[REGS];
  __device__ void init_reads(int f0) {
    const int lane = threadIdx.x & 63;
    if constexpr (KC) {
      const int row = f0 + (lane & 31);
#pragma unroll
      for (int ks = 0; ks < 2; ks++) at[ks] = row * 64 + (((2 * ks + (lane >> 5)) ^ swz(row)) << 4);
    } else {
      const int G = lane >> 4, j = lane & 15;
      const int row = 8 * (G >> 1) + (j >> 2);  // + 4 * half + 16 * ks: the same swizzle
#pragma unroll
      for (int b = 0; b < REGS; b++) {
        const int c = (f0 >> 3) + 4 * b + 2 * (G & 1) + ((j & 3) >> 1);
        at[b] = row * (F * 2) + ((c ^ swz(row)) << 4) + ((j & 1) << 3);
      }
    }
  }
  __device__ void read(char* lds, int b, int ks, int half, bf16x8& f) const {
    if constexpr (KC) {
      f = *(const bf16x8*)(lds + at[ks] + b * 2048);
    } else {
      // The swizzle changes the chunk's bits 2 and 3 (F = 64: bit 2): blocks
      // that differ above them are a constant apart.
      const bf16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_bf16x4*)((lds_char*)lds + at[b % REGS] + (b / REGS) * (REGS * 64) + (16 * ks + 4 * half) * (F * 2)));
#pragma unroll
      for (int i = 0; i < 4; i++) f[4 * half + i] = x[i];
    }
  }
};

template <typename TO>
__device__ inline void store_tail(TO* o, const float* v, int n, bool add) {
#pragma unroll
  for (int i = 0; i < 7; i++)
    if (i < n) {
      if constexpr (sizeof(TO) == 4)
        o[i] = add ? o[i] + v[i] : v[i];
      else
        o[i] = (uint16_t)dev::bf16_rne(add ? dev::bf16_to_f32(o[i]) + v[i] : v[i]);
    }
}

template <typename TO, int FORM, int NB, int NS, bool DMA>
__global__ __launch_bounds__(THREADS, NB == 8 ? 1 : 2) void expert_mfma_kernel(const ExpertArgs a) {
  constexpr int BN = 32 * NB;
  using FeedA = Feed<FORM == EXPERT_AK, BM, DMA>;
  using FeedB = Feed<FORM != EXPERT_DW, BN, DMA>;
  constexpr int PER_STEP = FeedA::N + FeedB::N;
  constexpr int BBASE = NS * FeedA::BYTES;
  __shared__ __attribute__((aligned(1024))) char smem[NS * (FeedA::BYTES + FeedB::BYTES)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  FeedA fa;
  FeedB fb;
  TO* out;
  int K, mrows, nrows;
  if constexpr (FORM == EXPERT_DW) {
    const dev::ExpertTile t = dev::find_weight_tile(a, blockIdx.x);
    K = t.end - t.begin;
    if (a.accumulate && K == 0) return;
    const int m0 = t.m_tile * BM, n0 = t.n_tile * BN;
    mrows = a.M - m0;
    nrows = a.N - n0;
    fa.init((const uint16_t*)a.a + t.begin * a.lda + m0, a.lda, mrows, K);
    fb.init((const uint16_t*)a.b + t.begin * a.ldb + n0, a.ldb, nrows, K);
    out = (TO*)a.out + t.e * a.o_expert + n0 * a.ldo + m0;
  } else {
    const dev::ExpertTile t = dev::find_row_tile(a, blockIdx.x, BN);
    if (!t.ok) return;
    K = t.e < a.E ? a.K : 0;  // rows past the last expert's: zeros
    const int n0 = t.begin + t.n_tile * BN, m0 = t.m_tile * BM;
    mrows = a.M - m0;
    nrows = t.end - n0;
    fa.init((const uint16_t*)a.a + (t.e < a.E ? t.e * a.a_expert : 0) + (FORM == EXPERT_AK ? m0 * a.lda : (int64_t)m0),
            a.lda, mrows, K);
    fb.init((const uint16_t*)a.b + n0 * a.ldb, a.ldb, nrows, K);
    out = (TO*)a.out + n0 * a.ldo + m0;
  }
  fa.init_reads(64 * wave);
  fb.init_reads(0);
  const int KT = __builtin_amdgcn_readfirstlane((K + BK - 1) / BK);

  f32x16 acc[2][NB];
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int j = 0; j < NB; j++)
#pragma unroll
      for (int v = 0; v < 16; v++) acc[i][j][v] = 0.f;

  const uint32_t smem_base = (uint32_t)(uintptr_t)(lds_char*)smem;
  const uint32_t ma = __builtin_amdgcn_readfirstlane(smem_base + (uint32_t)(wave * FeedA::N * 1024));
  const uint32_t mb = __builtin_amdgcn_readfirstlane(smem_base + (uint32_t)(BBASE + wave * FeedB::N * 1024));
  auto issue_a = [&](int stage, int i) { fa.issue(i, ma + (uint32_t)(stage * FeedA::BYTES + i * 1024)); };
  auto issue_b = [&](int stage, int i) { fb.issue(i, mb + (uint32_t)(stage * FeedB::BYTES + i * 1024)); };

  // The main loop over L of the NB row blocks.
  auto product = [&](auto lc) {
    constexpr int L = decltype(lc)::value;
    constexpr int Q = 2 * L;                                         // MFMAs of 16 k
    constexpr int R = 2 * FeedA::READS + L * FeedB::READS;           // fragment reads of 16 k
    bf16x8 a0[2], a1[2], b0[L], b1[L];
    auto read_one = [&](int stage, int ks, int r, bf16x8 (&ra)[2], bf16x8 (&rb)[L]) {
      if (r < 2 * FeedA::READS)
        fa.read(smem + stage * FeedA::BYTES, r / FeedA::READS, ks, r % FeedA::READS, ra[r / FeedA::READS]);
      else {
        const int s = r - 2 * FeedA::READS;
        fb.read(smem + BBASE + stage * FeedB::BYTES, s / FeedB::READS, ks, s % FeedB::READS, rb[s / FeedB::READS]);
      }
    };
    if constexpr (DMA) {
      // 16 k: MFMAs on (xa, xb), reading (ya, yb) of the next 16 k and
      // issuing an operand's loads in between.  The order is pinned: a wave
      // issues an instruction every four clocks at most, and an MFMA takes 32.
      auto half = [&](const bf16x8 (&xa)[2], const bf16x8 (&xb)[L], int stage, int ks, bf16x8 (&ya)[2],
                      bf16x8 (&yb)[L], int loads, auto&& load, auto&& step) {
#pragma unroll
        for (int q = 0; q < Q; q++) {
          const int n = q >> 1, m = (n & 1) ? 1 - (q & 1) : q & 1;
          acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[m], xb[n], acc[m][n], 0, 0, 0);
#pragma unroll
          for (int r = q * R / Q; r < (q + 1) * R / Q; r++) read_one(stage, ks, r, ya, yb);
#pragma unroll
          for (int i = q * loads / Q; i < (q + 1) * loads / Q; i++) load(i);
          if (q == Q - 1) step();
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      // Step kt: during its first 16 k the rows of step kt + NS - 1 are
      // loaded; then, once step kt + 1 has landed and every wave has read
      // step kt's second 16 k (barrier), its stage takes step kt + NS's
      // features.  Ahead of the loop: steps 0 .. NS - 2 and the features of
      // step NS - 1.
#pragma unroll
      for (int s = 0; s < NS; s++) {
#pragma unroll
        for (int i = 0; i < FeedA::N; i++) issue_a(s, i);
        fa.advance(s + 1, KT);
        if (s < NS - 1) {
#pragma unroll
          for (int i = 0; i < FeedB::N; i++) issue_b(s, i);
          fb.advance(s + 1, KT);
        }
      }
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((NS - 2) * PER_STEP + FeedA::N));
      __builtin_amdgcn_s_barrier();
#pragma unroll
      for (int r = 0; r < R; r++) read_one(0, 0, r, a0, b0);
      auto iter = [&](int kt, auto sc) {
        constexpr int S = decltype(sc)::value;
        half(a0, b0, S, 1, a1, b1, FeedB::N, [&](int i) { issue_b((S + NS - 1) % NS, i); },
             [&]() { fb.advance(kt + NS, KT); });
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((NS - 2) * PER_STEP));
        __builtin_amdgcn_s_barrier();
        half(a1, b1, (S + 1) % NS, 0, a0, b0, FeedA::N, [&](int i) { issue_a(S, i); },
             [&]() { fa.advance(kt + NS + 1, KT); });
      };
#pragma unroll 1
      for (int kt = 0; kt < KT; kt += NS) {
        iter(kt, std::integral_constant<int, 0>());
        if (kt + 1 < KT) iter(kt + 1, std::integral_constant<int, 1>());
        if (kt + 2 < KT) iter(kt + 2, std::integral_constant<int, 2>());
        if constexpr (NS > 3)
          if (kt + 3 < KT) iter(kt + 3, std::integral_constant<int, 3>());
      }
      // Loads past the last step (zeros) land before the stages are reused.
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
      __syncthreads();
    } else {
      fa.load(0);
      fb.load(0);
      fa.stage(smem);
      fb.stage(smem + BBASE);
      fa.load(1);
      fb.load(1);
      auto iter = [&](int kt, auto sc) {
        constexpr int S = decltype(sc)::value;
        // Stage S is filled, and everyone has read stage 1 - S.
        __syncthreads();
        fa.stage(smem + (1 - S) * FeedA::BYTES);
        fb.stage(smem + BBASE + (1 - S) * FeedB::BYTES);
        fa.load(kt + 2);
        fb.load(kt + 2);
#pragma unroll
        for (int r = 0; r < R; r++) read_one(S, 0, r, a0, b0);
#pragma unroll
        for (int r = 0; r < R; r++) read_one(S, 1, r, a1, b1);
#pragma unroll
        for (int q = 0; q < Q; q++)
          acc[q & 1][q >> 1] =
              __builtin_amdgcn_mfma_f32_32x32x16_bf16(a0[q & 1], b0[q >> 1], acc[q & 1][q >> 1], 0, 0, 0);
#pragma unroll
        for (int q = 0; q < Q; q++)
          acc[q & 1][q >> 1] =
              __builtin_amdgcn_mfma_f32_32x32x16_bf16(a1[q & 1], b1[q >> 1], acc[q & 1][q >> 1], 0, 0, 0);
      };
#pragma unroll 1
      for (int kt = 0; kt < KT; kt += 2) {
        iter(kt, std::integral_constant<int, 0>());
        if (kt + 1 < KT) iter(kt + 1, std::integral_constant<int, 1>());
      }
      __syncthreads();
    }
  };
  if (KT > 0) {
    if (NB <= 2 || nrows > 32 * (NB - 2)) {
      product(std::integral_constant<int, NB>());
    } else if (NB <= 4 || nrows > 32 * (NB - 4)) {
      product(std::integral_constant<int, (NB > 2 ? NB - 2 : NB)>());
    } else if (nrows > 64) {
      product(std::integral_constant<int, (NB > 4 ? 4 : NB)>());
    } else {
      product(std::integral_constant<int, 2>());
    }
  }

  // ---- results: block n of a wave (32 rows x 64 features) through its own
  // staging buffer, then 128 bytes (f32: 256) of a row by 8 (16) lanes.  dW is
  // staged in f32, since a value that is accumulated is rounded after the sum.
  // A lane holds row lane % 32, features 32 m + 8 q + 4 (lane / 32) + 0..3.
  constexpr bool WIDE = FORM == EXPERT_DW;
  constexpr int SROW = WIDE ? 256 : 128;
  constexpr int SBUF = WIDE ? 1 : 2;
  static_assert(4 * 32 * SROW * SBUF <= (int)sizeof(smem), "staging fits the stages");
  const int fm = 64 * wave;
  if (fm >= mrows) return;
  char* const st0 = smem + wave * (SBUF * 32 * SROW);
#pragma unroll
  for (int n = 0; n < NB; n++) {
    if (32 * n >= nrows) break;
    char* const st = st0 + (n % SBUF) * (32 * SROW);
    const int r = lane & 31;
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const f32x16& c = acc[m][n];
        if constexpr (WIDE) {
          const int chunk = 8 * m + 2 * q + (lane >> 5);
          *(f32x4*)(st + r * SROW + ((chunk ^ (r & 15)) << 4)) =
              f32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
        } else {
          const int chunk = 4 * m + q;
          *(u32x2*)(st + r * SROW + ((chunk ^ (r & 7)) << 4) + ((lane >> 5) << 3)) =
              u32x2{dev::bf16_pack2(c[4 * q], c[4 * q + 1]), dev::bf16_pack2(c[4 * q + 2], c[4 * q + 3])};
        }
      }
    asm volatile("" ::: "memory");  // a wave's LDS accesses run in order
    if constexpr (!WIDE) {
#pragma unroll
      for (int it = 0; it < 4; it++) {
        const int row = 8 * it + (lane >> 3), c = lane & 7;
        const u32x4 v = *(const u32x4*)(st + row * SROW + ((c ^ (row & 7)) << 4));
        const int left = mrows - fm - 8 * c;
        if (32 * n + row < nrows) {
          uint16_t* o = (uint16_t*)out + (32 * n + row) * a.ldo + fm + 8 * c;
          if (left >= 8) {
            *(u32x4u*)o = v;
          } else {
#pragma unroll
            for (int i = 0; i < 7; i++)
              if (i < left) o[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
          }
        }
      }
    } else if constexpr (sizeof(TO) == 4) {
#pragma unroll
      for (int it = 0; it < 8; it++) {
        const int row = 4 * it + (lane >> 4), c = lane & 15;
        f32x4 v = *(const f32x4*)(st + row * SROW + ((c ^ (row & 15)) << 4));
        const int left = mrows - fm - 4 * c;
        if (32 * n + row < nrows) {
          float* o = (float*)out + (32 * n + row) * a.ldo + fm + 4 * c;
          if (left >= 4) {
            if (a.accumulate) v += *(const f32x4u*)o;
            *(f32x4u*)o = v;
          } else {
            store_tail(o, (const float*)&v, left, a.accumulate);
          }
        }
      }
    } else {
#pragma unroll
      for (int it = 0; it < 4; it++) {
        const int row = 8 * it + (lane >> 3), c = lane & 7;
        float v[8];
        *(f32x4*)v = *(const f32x4*)(st + row * SROW + (((2 * c) ^ (row & 15)) << 4));
        *(f32x4*)(v + 4) = *(const f32x4*)(st + row * SROW + (((2 * c + 1) ^ (row & 15)) << 4));
        const int left = mrows - fm - 8 * c;
        if (32 * n + row < nrows) {
          uint16_t* o = (uint16_t*)out + (32 * n + row) * a.ldo + fm + 8 * c;
          if (left >= 8) {
            if (a.accumulate) {
              const u32x4 old = *(const u32x4u*)o;
#pragma unroll
              for (int i = 0; i < 8; i++) v[i] += dev::bf16_to_f32((old[i >> 1] >> (16 * (i & 1))) & 0xffffu);
            }
            *(u32x4u*)o = u32x4{dev::bf16_pack2(v[0], v[1]), dev::bf16_pack2(v[2], v[3]),
                                dev::bf16_pack2(v[4], v[5]), dev::bf16_pack2(v[6], v[7])};
          } else {
            store_tail(o, v, left, a.accumulate);
          }
        }
      }
    }
    asm volatile("" ::: "memory");
  }
}

template <typename TO, int FORM>
const void* pick(int bn, bool dma) {
  if (bn == 256)
    return dma ? (const void*)&expert_mfma_kernel<TO, FORM, 8, 4, true>
               : (const void*)&expert_mfma_kernel<TO, FORM, 8, 2, false>;
  return dma ? (const void*)&expert_mfma_kernel<TO, FORM, 4, 3, true>
             : (const void*)&expert_mfma_kernel<TO, FORM, 4, 2, false>;
}

}  // namespace

int launch_expert_mfma(const ExpertArgs& a, const ExpertLaunch& l, void* stream) {
  const void* k = l.form == EXPERT_AK   ? pick<uint16_t, EXPERT_AK>(l.bn, l.dma)
                  : l.form == EXPERT_AM ? pick<uint16_t, EXPERT_AM>(l.bn, l.dma)
                  : l.out_dtype == CBD_F32 ? pick<float, EXPERT_DW>(l.bn, l.dma)
                                           : pick<uint16_t, EXPERT_DW>(l.bn, l.dma);
  void* args[] = {const_cast<ExpertArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
