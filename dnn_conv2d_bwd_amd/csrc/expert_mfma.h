// expert_mfma.h -- bf16 expert products with many rows, on
// v_mfma_f32_32x32x16_bf16.
//
// A workgroup of 4 waves (2 x 2) computes 64 * MB features (m, the contiguous
// side of the output) x 64 * NB rows (n) of one expert in steps of 64 k (dW: 32).
// Waves own half the features each and take turns in the 32-row blocks, so a tile
// that the expert's rows do not fill costs matrix time only for the 64 rows it
// has begun, the same for every wave; and a wave's results leave through a
// staging buffer of its own without a barrier.
//
// Workgroups stay: each takes tiles b, b + grid, ... and issues the first loads
// of its next tile before it writes the results of the last one, which then
// leave while the next tile's products run.
//
// Operand tiles go into two (dW: four) LDS stages.  DMA: buffer_load ... lds,
// 16 bytes a lane, issued between the MFMAs of a step's first and last 16 k, one
// barrier a step; the reads of the next 16 k are spread between the MFMAs.
// Without DMA (rows off 16-byte alignment, or a contracted length that is no
// multiple of 8 where k is contiguous): through registers, one step ahead.
// What is past the contracted length is zero in both operands, and what rows
// and features past the other edges give is not stored, so nothing beyond the
// rows of an expert or the contracted length takes part.
//
// A step is 64 k, since a k-contiguous row is then fetched in whole 128-byte
// lines: with 32 k (64 bytes) the L2s' requests, one a clock and channel, take
// as long as the MFMAs (256 x 256 tile: 16384 per step and XCD over 16
// channels = 1024 clocks).
//
// A k-contiguous operand is staged [row][64 k], chunk c (16 bytes) of row r at
// c ^ (r / 2 % 8), and read with ds_read_b128.  A feature-contiguous one is
// staged [k][features] and read with ds_read_b64_tr_b16, which hands lane j of
// 16 the four k of feature j; its chunks are moved by 64 bytes a row so that
// the four k rows of a read sit in different banks.
//
// Bound: with random bf16 values the card's power (a loop of nothing but these
// MFMAs runs at 1.89 PFLOP/s) and, below that, the loads: at a full clock
// (zeros) a 65536 x 8192 x 2048 product takes 1.48 ms, 1.49 without the LDS
// reads, 1.19 with every load an L2 hit and 0.98 without the loads.  Measured:
// 65536 x 4096 x 2048, 32 experts, forward 0.93 ms (1.18 PFLOP/s), weight
// gradient in f32 1.1 ms (1.0 PFLOP/s); 16384 x 2048 x 1408, 64 experts, data
// gradient 132 us (3.6 TB/s, 0.71 PFLOP/s).
//
// Gated forward, a wave's features are half the gate's and half the same ones of
// the other projection (dev::Pair), so that a lane ends with both and their
// product never leaves it; the workgroup's loads take the two places of W in
// turn.  32768 x 4096 x 2 x 2048, 32 experts: 935 - 953 us, as the plain product
// of 65536 x 4096 x 2048 needs; 993 - 1016 with both projections saved (268 MB
// more to write while the next tile's products run); matrix units busy 61 % of the
// clocks, the rest as above.  Gated backward, the tile's gates are read where its
// results go: 128 wide ahead of the last step's products (1408 outputs x 2048, 64
// experts, 16384 rows: 168 us, 772 MB moved at 4.6 TB/s; the plain product, which
// has 184 MB less to move, 130), 256 wide block by block, for want of registers.
//
// Two stages of 64 k against four of 32 k (dW has no k-contiguous operand, so
// its lines are whole either way): dW 1130 / 1100 us, 64 experts of 1408
// outputs and 1024 rows each 443 / 476 us.
#pragma once
#include <type_traits>

#include "cbd_device.h"
#include "expert_device.h"
#include "gate_device.h"

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

constexpr int THREADS = 256;
// Cache policy of the results' stores: non-temporal (64 experts' 2048 x 1408
// f32 gradients from 256 rows each 220 -> 165 us, 16384 x 64 x 2048 x 1408
// data gradient 137 -> 134 us).
constexpr int kStoreAux = 2;

// s_waitcnt immediate: vmcnt <= n (at most 63), lgkmcnt 0 (gfx9 encoding).
constexpr int waitcnt_vm_lgkm0(int n) {
  n = n > 63 ? 63 : n;
  return (n & 15) | (7 << 4) | ((n >> 4) << 14);
}

// The thread's index, opaque: what is computed from it once a tile is not kept
// in registers through the main loop.
__device__ inline int fresh_tid() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// One operand: F features (or rows) by BK k a stage; the 32-row blocks that a
// wave reads are EVERY blocks apart.  PAIR: of two projections whose features
// lie `up` elements apart (dev::Pair), `rows` counting those of one.
template <bool KC, int F, int BK, int EVERY, bool DMA, bool PAIR = false>
struct Feed {
  static constexpr int BYTES = F * BK * 2;
  static constexpr int N = BYTES / 4096;  // 1 KiB blocks a wave fills
  static constexpr int CHUNKS = (KC ? BK : F) / 8;  // 16-byte chunks of a row

  __device__ static int swz(int row) {
    return KC ? (BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3) : 4 * (row & 3);
  }
  // Row (KC: of features; else of k) and chunk that a lane fills of block i.
  CBD_INLINE __device__ static int fill_row(int i, int tid) {
    const int lane = tid & 63, j = N * (tid >> 6) + i;
    return (64 / CHUNKS) * j + lane / CHUNKS;
  }
  CBD_INLINE __device__ static int fill_chunk(int i, int tid) {
    const int lane = tid & 63;
    return (lane % CHUNKS) ^ swz(fill_row(i, tid));
  }

  // Feature (or row) of the operand that row r of the tile holds, and whether
  // it is the second projection's.
  __device__ static int feat(int r) { return PAIR ? dev::Pair<F, 2>::feat(r) : r; }
  __device__ static int part(int r) { return PAIR ? dev::Pair<F, 2>::part(r) : 0; }
  static constexpr int FEATS = PAIR ? F / 2 : F;

  const uint16_t* p;  // element (row 0, k 0)
  int64_t ld;
  int rows, K;        // features inside the operand; contracted length
  // DMA
  uint32_t voff[N];
  uint32_t soff, rec, step;
  int64_t left;       // feature-contiguous: bytes from the next step's first k row to the end
  uint64_t base;
  // registers: the lane's 16 bytes of each block, where the next step's are
  // and, feature-contiguous, the features from there to the edge
  u32x4 v[N];
  const uint16_t* q[N];
  int feats[N];
  bool wide;    // 8 elements or more in a row of the operand
  bool inside;  // every chunk of the wave's is loaded whole
  bool edge;    // some of them from `back` features further down
  int back[N];

  // width: of the whole operand's features.
  CBD_INLINE __device__ void init(const uint16_t* p_, int64_t ld_, int rows_, int K_, int width, int64_t up = 0) {
    wide = (KC ? K_ : width) >= 8;
    p = p_;
    ld = ld_;
    rows = rows_;
    K = K_;
    if constexpr (DMA) {
      base = dev::uniform((uint64_t)p);
      soff = 0;
      step = (uint32_t)(BK * ld * 2);
      left = K > 0 ? ((int64_t)(K - 1) * ld + rows + (PAIR ? up : 0)) * 2 : 0;
      const int tid = fresh_tid();
#pragma unroll
      for (int i = 0; i < N; i++) {
        const int r = fill_row(i, tid), c = fill_chunk(i, tid);
        if constexpr (PAIR) {
          const int f = feat(KC ? r : 8 * c);
          const uint32_t at = KC ? (uint32_t)f * (uint32_t)ld * 2u + (uint32_t)c * 16u
                                 : (uint32_t)r * (uint32_t)ld * 2u + (uint32_t)f * 2u;
          voff[i] = f < rows ? at + (uint32_t)part(KC ? r : 8 * c) * (uint32_t)up * 2u : dev::kOOB;
        } else {
          voff[i] = (KC ? r < rows : 8 * c < rows) ? (uint32_t)r * (uint32_t)ld * 2u + (uint32_t)c * 16u : dev::kOOB;
        }
      }
      if constexpr (KC) {
        rec = K > 0 ? (uint32_t)(((int64_t)((rows < FEATS ? rows : FEATS) - 1) * ld + (PAIR ? up : 0) + K) * 2) : 0u;
        mask_tail(0);
      } else {
        clamp();
      }
    } else {
      const int tid = fresh_tid();
      inside = true;
      edge = false;
#pragma unroll
      for (int i = 0; i < N; i++) {
        const int r = fill_row(i, tid), c = 8 * fill_chunk(i, tid);
        if (KC) {
          const int f = feat(r);
          q[i] = p + (f < rows ? f : rows - 1) * ld + c;
          if (PAIR) q[i] += part(r) * up;
        } else {
          const int f = feat(c) < rows ? feat(c) : 0;
          q[i] = p + r * ld + f;
          if (PAIR) q[i] += part(c) * up;
          feats[i] = rows - f;
          // A chunk that passes the edge is loaded from further down, and
          // moved when it is staged: no wait for it here.
          back[i] = feats[i] < 8 && wide ? 8 - feats[i] : 0;
          if (back[i]) {
            q[i] -= back[i];
            feats[i] = 8;
          }
          edge = edge || __any(back[i] != 0);
          inside = inside && __all(feats[i] >= 8);
        }
      }
    }
  }
  // Step t is the last and part of its k are past the end.
  CBD_INLINE __device__ void mask_tail(int t) {
    const int over = K - t * BK;
    if (over < BK) {
      const int tid = fresh_tid();
#pragma unroll
      for (int i = 0; i < N; i++)
        if (8 * fill_chunk(i, tid) >= over) voff[i] = dev::kOOB;
    }
  }
  CBD_INLINE __device__ void clamp() {
    const int64_t l = (left + 3) & ~(int64_t)3;
    rec = left <= 0 ? 0u : l > 0x7ffffffc ? 0x7ffffffcu : (uint32_t)l;
  }
  // To step t (of steps); past the last the record count is 0.
  CBD_INLINE __device__ void advance(int t, int steps) {
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
  CBD_INLINE __device__ void issue(int i, uint32_t m0v) const {
    const i32x4 d = {(int)(uint32_t)base, (int)((uint32_t)(base >> 32) & 0xffffu), (int)rec, 0x00020000};
    const uint32_t so = KC ? soff : 0u;
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds\n\ts_nop 0"
                 ::"s"(m0v), "v"(voff[i]), "s"(d), "s"(so) : "memory", "m0");
#pragma clang diagnostic pop
  }

  // y moved down by n < 8 elements.
  CBD_INLINE __device__ static u32x4 down(u32x4 y, int n) {
    uint64_t lo = (uint64_t)y[1] << 32 | y[0], hi = (uint64_t)y[3] << 32 | y[2];
    if (n >= 4) {
      lo = hi;
      hi = 0;
      n -= 4;
    }
    const int by = 16 * n;  // 0, 16, 32 or 48
    lo = by > 0 ? lo >> by | hi << (64 - by) : lo;
    hi >>= by;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
  // The first n < 8 elements from s, zeros after them: by elements, or the 16
  // bytes that end with them, moved down.
  CBD_INLINE __device__ u32x4 first(const uint16_t* s, int n) const {
    if (KC && wide) return down(*(const u32x4u*)(s - (8 - n)), 8 - n);
    u32x4 x = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 7; j++)
      if (j < n) x[j >> 1] |= (uint32_t)s[j] << (16 * (j & 1));
    return x;
  }
  // Through registers: the next step, of which `left` k are inside, zeros past
  // them.  Rows and features past an edge repeat others; what they give is not
  // stored.
  CBD_INLINE __device__ void load(int left) {
    if (left >= BK && inside) {
#pragma unroll
      for (int i = 0; i < N; i++) {
        v[i] = *(const u32x4u*)q[i];
        q[i] += KC ? BK : BK * ld;
      }
      return;
    }
    const int tid = fresh_tid();
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int k = KC ? 8 * fill_chunk(i, tid) : fill_row(i, tid);
      const int n = KC ? left - k : k < left ? feats[i] : 0;
      u32x4 x = {0u, 0u, 0u, 0u};
      if (n >= 8)
        x = *(const u32x4u*)q[i];
      else if (n > 0)
        x = first(q[i], n);
      v[i] = x;
      q[i] += KC ? BK : BK * ld;
    }
  }
  CBD_INLINE __device__ void stage(char* lds) const {
#pragma unroll
    for (int i = 0; i < N; i++)
      *(u32x4*)(lds + (N * (int)(threadIdx.x >> 6) + i) * 1024 + (threadIdx.x & 63) * 16) =
          !KC && edge ? down(v[i], back[i]) : v[i];
  }

  // ---- fragments: of 32 rows (block b from feature f0), 16 k (step ks).
  static constexpr int READS = KC ? 1 : 2;  // LDS reads a fragment takes
  static constexpr int REGS = KC ? BK / 16 : 4 / EVERY;
  int at[REGS];
  CBD_INLINE __device__ void init_reads(int f0) {
    const int lane = threadIdx.x & 63;
    if constexpr (KC) {
      const int row = f0 + (lane & 31);
#pragma unroll
      for (int ks = 0; ks < BK / 16; ks++) at[ks] = row * (BK * 2) + (((2 * ks + (lane >> 5)) ^ swz(row)) << 4);
    } else {
      const int G = lane >> 4, j = lane & 15;
      const int row = 8 * (G >> 1) + (j >> 2);  // + 4 * half + 16 * ks: the same swizzle
#pragma unroll
      for (int b = 0; b < REGS; b++) {
        const int c = (f0 >> 3) + 4 * EVERY * b + 2 * (G & 1) + ((j & 3) >> 1);
        at[b] = row * (F * 2) + ((c ^ swz(row)) << 4) + ((j & 1) << 3);
      }
    }
  }
  CBD_INLINE __device__ void read(char* lds, int b, int ks, int half, bf16x8& f) const {
    if constexpr (KC) {
      f = *(const bf16x8*)(lds + at[ks] + b * (EVERY * 64 * BK));
    } else {
      // The swizzle changes the chunk's bits 2 and 3: blocks that differ above
      // them are a constant apart.
      const bf16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_bf16x4*)((lds_char*)lds + at[b % REGS] + (b / REGS) * (REGS * EVERY * 64) + (16 * ks + 4 * half) * (F * 2)));
#pragma unroll
      for (int i = 0; i < 4; i++) f[4 * half + i] = x[i];
    }
  }
};

// How results are written: in whole 16-byte chunks on their boundaries; those
// added to what is there; or at any alignment and width, added or not.
enum Out { WHOLE, WHOLE_ADD, ANY };

// A gated tile's first feature and row.
struct Where {
  int m0, n0;
};
struct Nowhere {};

template <typename TO, int FORM, int MB, int NB, bool DMA, Out OUT, int GATE = GATE_NONE>
__global__ __launch_bounds__(THREADS, MB == 4 ? 1 : 2) void expert_mfma_kernel(
    const std::conditional_t<GATE == GATE_NONE, ExpertArgs, GatedArgs> a) {
  constexpr int BM = 64 * MB, BN = 64 * NB;
  constexpr bool PAIR = GATE == GATE_FWD || GATE == GATE_FWD_SAVE;
  constexpr int FEATS = PAIR ? BM / 2 : BM;  // features of the output that a tile has
  // Two stages of 64 k, or four of 32.
  constexpr int BK = FORM != EXPERT_DW ? 64 : 32, NS = 128 / BK;
  using FeedA = Feed<FORM == EXPERT_AK, BM, BK, 1, DMA, PAIR>;
  using FeedB = Feed<FORM != EXPERT_DW, BN, BK, 2, DMA>;
  using Tiles = std::conditional_t<FORM == EXPERT_DW, dev::WeightTiles, dev::RowTiles>;
  constexpr int BBASE = NS * FeedA::BYTES;
  constexpr int STAGES = BBASE + NS * FeedB::BYTES;
  // Results of a wave leave through SBUF buffers of 32 rows x 128 bytes.
  constexpr int SBUF = MB == 4 ? 2 : 1;
  __shared__ __attribute__((aligned(1024))) char smem[STAGES + 4 * SBUF * 4096];
  // 32-feature blocks of a buffer; what is added to is staged in f32 and rounded after the sum.
  constexpr bool F32 = sizeof(TO) == 4 || OUT == WHOLE_ADD;
  constexpr int HM = F32 ? 1 : 2;
  // Stores of a wave's whole tile.
  constexpr int STORES = GATE == GATE_NONE ? NB * (MB / HM) * 4 : PAIR ? NB * MB * (GATE == GATE_FWD ? 1 : 3) : 0;
  const int wave = threadIdx.x >> 6, wm = wave & 1, wn = wave >> 1;

  const uint32_t smem_base = (uint32_t)(uintptr_t)(lds_char*)smem;
  const uint32_t ma = __builtin_amdgcn_readfirstlane(smem_base + (uint32_t)(wave * FeedA::N * 1024));
  const uint32_t mb = __builtin_amdgcn_readfirstlane(smem_base + (uint32_t)(BBASE + wave * FeedB::N * 1024));
  FeedA fa;
  FeedB fb;
  fa.init_reads(32 * MB * wm);
  fb.init_reads(32 * wn);
  auto issue_a = [&](int stage, int i) CBD_INLINE { fa.issue(i, ma + (uint32_t)(stage * FeedA::BYTES + i * 1024)); };
  auto issue_b = [&](int stage, int i) CBD_INLINE { fb.issue(i, mb + (uint32_t)(stage * FeedB::BYTES + i * 1024)); };

  // A tile: its contracted length, and where and how much it writes.
  struct Tile : std::conditional_t<GATE == GATE_NONE, Nowhere, Where> {
    TO* out;
    int K, mrows, nrows;
  };
  // Points the feeds at tile t and issues its first loads: of NS steps, but
  // with more than two stages not the rows of the last.
  auto begin = [&](const dev::ExpertTile& t) CBD_INLINE -> Tile {
    Tile c;
    const int m0 = t.m_tile * FEATS;
    c.mrows = a.M - m0;
    if constexpr (FORM == EXPERT_DW) {
      const int n0 = t.n_tile * BN;
      c.K = t.end - t.begin;
      c.nrows = a.N - n0;
      fa.init((const uint16_t*)a.a + t.begin * a.lda + m0, a.lda, c.mrows, c.K, a.M);
      fb.init((const uint16_t*)a.b + t.begin * a.ldb + n0, a.ldb, c.nrows, c.K, a.N);
      c.out = (TO*)a.out + t.e * a.o_expert + n0 * a.ldo + m0;
    } else {
      const int n0 = t.begin;
      c.K = t.e < a.E ? a.K : 0;  // rows past the last expert's: zeros
      c.nrows = t.end - n0;
      fa.init((const uint16_t*)a.a + (t.e < a.E ? t.e * a.a_expert : 0) +
                  (FORM == EXPERT_AK ? m0 * a.lda : (int64_t)m0),
              a.lda, c.mrows, c.K, a.M, [&] {
                if constexpr (PAIR)
                  return a.up;
                else
                  return (int64_t)0;
              }());
      fb.init((const uint16_t*)a.b + n0 * a.ldb, a.ldb, c.nrows, c.K, a.N);
      c.out = (TO*)a.out + n0 * a.ldo + m0;
      if constexpr (GATE != GATE_NONE) {
        c.m0 = m0;
        c.n0 = n0;
      }
    }
    if constexpr (DMA) {
      const int steps = (c.K + BK - 1) / BK;
#pragma unroll
      for (int s = 0; s < NS; s++) {
#pragma unroll
        for (int i = 0; i < FeedA::N; i++) issue_a(s, i);
        fa.advance(s + 1, steps);
        if (NS > 2 && s == NS - 1) break;
#pragma unroll
        for (int i = 0; i < FeedB::N; i++) issue_b(s, i);
        fb.advance(s + 1, steps);
      }
    } else {
      fa.load(c.K);
      fb.load(c.K);
    }
    return c;
  };

  bool deep = false;  // a whole tile's stores were issued after this tile's first loads

  // Results: HM blocks of 32 features of a 32-row block at a time through one
  // of the wave's buffers, then 128 bytes of a row by 8 lanes.  A lane of a
  // block holds row lane % 32, features 8 q + 4 (lane / 32) + 0..3.
  auto finish = [&](const Tile& c, auto lc, f32x16 (&acc)[MB][decltype(lc)::value]) CBD_INLINE {
    constexpr int L = decltype(lc)::value;
    const int tid = fresh_tid(), lane = tid & 63;
    const int wm = (tid >> 6) & 1, wn = tid >> 7;
    char* const st0 = smem + STAGES + (tid >> 6) * (SBUF * 4096);
    const auto ro = dev::rsrc(c.out, 0x7ffffffcu);
    const int r = lane & 31, hi = lane >> 5;
#pragma unroll
    for (int i = 0; i < L * (MB / HM); i++) {
      const int n = i / (MB / HM), h = i % (MB / HM);
      const int fm = 32 * MB * wm + 32 * HM * h, rn = 64 * n + 32 * wn;
      char* const st = st0 + (i % SBUF) * 4096;
      // The sums stay in accumulation registers until they are converted.
      if constexpr (MB == 4) {
#pragma unroll
        for (int m = 0; m < HM; m++) asm volatile("" : "+a"(acc[HM * h + m][n]));
      }
#pragma unroll
      for (int m = 0; m < HM; m++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; j++) v[j] = acc[HM * h + m][n][4 * q + j];
          if (OUT == ANY && FORM == EXPERT_DW && a.accumulate && rn + r < c.nrows) {
            const int f = fm + 32 * m + 8 * q + 4 * hi;
            const TO* o = c.out + (rn + r) * a.ldo + f;
#pragma unroll
            for (int j = 0; j < 4; j++)
              if (f + j < c.mrows) {
                if constexpr (sizeof(TO) == 4)
                  v[j] += o[j];
                else
                  v[j] += dev::bf16_to_f32(o[j]);
              }
          }
          if constexpr (F32)
            *(f32x4*)(st + r * 128 + (((2 * q + hi) ^ (r & 7)) << 4)) = v;
          else
            *(u32x2*)(st + r * 128 + (((4 * m + q) ^ (r & 7)) << 4) + (hi << 3)) =
                u32x2{dev::bf16_pack2(v[0], v[1]), dev::bf16_pack2(v[2], v[3])};
        }
      asm volatile("" ::: "memory");  // a wave's LDS accesses run in order
      constexpr int PER = F32 ? 4 : 8;  // elements of a chunk
#pragma unroll
      for (int it = 0; it < 4; it++) {
        const int row = 8 * it + (lane >> 3), ch = lane & 7;
        u32x4 v = *(const u32x4*)(st + row * 128 + ((ch ^ (row & 7)) << 4));
        const int f = fm + PER * ch;
        if constexpr (OUT != ANY) {
          // Past an edge: dropped.
          const uint32_t off = rn + row < c.nrows && f < c.mrows
                                   ? ((uint32_t)(rn + row) * (uint32_t)a.ldo + (uint32_t)f) * (uint32_t)sizeof(TO)
                                   : dev::kOOB;
          if constexpr (OUT == WHOLE_ADD && sizeof(TO) == 2) {
            const u32x2 old = __builtin_amdgcn_raw_buffer_load_b64(ro, off, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b64(
                u32x2{dev::bf16_pack2(__uint_as_float(v[0]) + dev::bf16_to_f32(old[0] & 0xffffu),
                                      __uint_as_float(v[1]) + __uint_as_float(old[0] & 0xffff0000u)),
                      dev::bf16_pack2(__uint_as_float(v[2]) + dev::bf16_to_f32(old[1] & 0xffffu),
                                      __uint_as_float(v[3]) + __uint_as_float(old[1] & 0xffff0000u))},
                ro, off, 0, kStoreAux);
          } else {
            if constexpr (OUT == WHOLE_ADD) {
              const u32x4 old = __builtin_amdgcn_raw_buffer_load_b128(ro, off, 0, 0);
#pragma unroll
              for (int j = 0; j < 4; j++) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(old[j]));
            }
            __builtin_amdgcn_raw_buffer_store_b128(v, ro, off, 0, kStoreAux);
          }
        } else if (rn + row < c.nrows) {
          TO* o = c.out + (rn + row) * a.ldo + f;
          if (c.mrows - f >= PER) {
            *(u32x4u*)o = v;
          } else {
#pragma unroll
            for (int j = 0; j < PER - 1; j++)
              if (f + j < c.mrows) {
                if constexpr (sizeof(TO) == 4)
                  o[j] = __uint_as_float(v[j]);
                else
                  o[j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
              }
          }
        }
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    }
    deep = OUT == WHOLE && L == NB;
  };

  // A chunk of N elements (8 or 4) of row `row`, feature f of a tile's part of
  // o; OUT == ANY: at any alignment and width.
  auto put = [&](const Tile& c, uint16_t* o, int64_t ld, int row, int f, auto v) CBD_INLINE {
    constexpr int N = sizeof(v) / 2;
    if constexpr (OUT != ANY) {
      const uint32_t off =
          row < c.nrows && f < c.mrows ? ((uint32_t)row * (uint32_t)ld + (uint32_t)f) * 2u : dev::kOOB;
      const auto r = dev::rsrc(o, 0x7ffffffcu);
      if constexpr (N == 8)
        __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, kStoreAux);
      else
        __builtin_amdgcn_raw_buffer_store_b64(v, r, off, 0, kStoreAux);
    } else if (row < c.nrows) {
      typedef uint32_t words __attribute__((ext_vector_type(N / 2), aligned(2)));
      uint16_t* const q = o + row * ld + f;
      if (c.mrows - f >= N) {
        *(words*)q = v;
      } else {
#pragma unroll
        for (int j = 0; j < N - 1; j++)
          if (f + j < c.mrows) q[j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
      }
    }
  };

  // Gated results.  Forward: a wave's blocks m are of the gate for m < MB / 2,
  // the others of the same features of the other projection; h and, saved, the
  // two leave one after another through the wave's buffer, HM blocks wide.
  // Backward: 16 rows by 64 features of dh at a time in f32, eight a lane, which
  // meet the same eight of g and u there.
  struct Gates {
    u32x4 g[4], u[4];  // of 32 rows by 64 features
  };
  [[maybe_unused]] auto fetch = [&](const Tile& c, int n, int h, Gates& x) CBD_INLINE {
    if constexpr (GATE == GATE_BWD) {
      const int tid = fresh_tid(), lane = tid & 63;
      const int wm = (tid >> 6) & 1, wn = tid >> 7;
      const uint16_t* const gs = (const uint16_t*)a.gu + c.n0 * a.ldgu + c.m0;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int row = 64 * n + 32 * wn + 8 * i + (lane >> 3), f = 32 * MB * wm + 64 * h + 8 * (lane & 7);
        if constexpr (OUT != ANY) {
          const uint32_t off = row < c.nrows && f < c.mrows ? ((uint32_t)row * (uint32_t)a.ldgu + (uint32_t)f) * 2u
                                                            : dev::kOOB;
          x.g[i] = __builtin_amdgcn_raw_buffer_load_b128(dev::rsrc(gs, 0x7ffffffcu), off, 0, kStoreAux);
          x.u[i] = __builtin_amdgcn_raw_buffer_load_b128(dev::rsrc(gs + a.M, 0x7ffffffcu), off, 0, kStoreAux);
        } else {
          x.g[i] = x.u[i] = u32x4{0u, 0u, 0u, 0u};
          if (row < c.nrows) {
            const uint16_t* const q = gs + row * a.ldgu + f;
            if (c.mrows - f >= 8) {
              x.g[i] = *(const u32x4u*)q;
              x.u[i] = *(const u32x4u*)(q + a.M);
            } else {
#pragma unroll
              for (int j = 0; j < 7; j++)
                if (f + j < c.mrows) {
                  x.g[i][j >> 1] |= (uint32_t)q[j] << (16 * (j & 1));
                  x.u[i][j >> 1] |= (uint32_t)q[a.M + j] << (16 * (j & 1));
                }
            }
          }
        }
      }
    }
  };
  // Units of 32 rows by 64 features, and how many of them have their gates
  // fetched ahead: all at the start of the main loop, or (256 x 256, and without
  // DMA: registers) one before the next tile's first loads, the others each a
  // unit before.
  constexpr int UNITS = MB / 2;
  [[maybe_unused]] constexpr bool EARLY = GATE == GATE_BWD && MB == 2 && DMA;
  [[maybe_unused]] auto finish_gated = [&](const Tile& c, auto lc, f32x16 (&acc)[MB][decltype(lc)::value],
                                           Gates (&ahead)[EARLY ? UNITS * decltype(lc)::value : 1]) CBD_INLINE {
    if constexpr (GATE != GATE_NONE) {
      constexpr int L = decltype(lc)::value;
      const int tid = fresh_tid(), lane = tid & 63;
      const int wm = (tid >> 6) & 1, wn = tid >> 7;
      char* const st0 = smem + STAGES + (tid >> 6) * (SBUF * 4096);
      const int r = lane & 31, hi = lane >> 5;
      if constexpr (PAIR) {
        constexpr int GM = MB / 2, CH = 4 * GM;   // blocks, and chunks of a row
        constexpr int OUTS = GATE == GATE_FWD ? 1 : 3;
        uint16_t* outs[OUTS];
        int64_t lds[OUTS];
        outs[0] = c.out;
        lds[0] = a.ldo;
        if constexpr (OUTS == 3) {
          outs[1] = (uint16_t*)a.gu + c.n0 * a.ldgu + c.m0;
          outs[2] = outs[1] + a.M;
          lds[1] = lds[2] = a.ldgu;
        }
#pragma unroll
        for (int n = 0; n < L; n++) {
#pragma unroll
          for (int o = 0; o < OUTS; o++) {
            char* const st = st0 + (SBUF == 2 && ((n * OUTS + o) & 1) ? 4096 : 0);
            // The sums stay in accumulation registers until they are converted.
            if constexpr (MB == 4) {
#pragma unroll
              for (int m = 0; m < MB; m++) asm volatile("" : "+a"(acc[m][n]));
            }
            auto stage = [&](auto&& value) CBD_INLINE {
#pragma unroll
              for (int m = 0; m < GM; m++)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                  float v[4];
#pragma unroll
                  for (int j = 0; j < 4; j++) v[j] = value(acc[m][n][4 * q + j], acc[m + GM][n][4 * q + j]);
                  *(u32x2*)(st + r * 128 + (((4 * m + q) ^ (r & 7)) << 4) + (hi << 3)) =
                      u32x2{dev::bf16_pack2(v[0], v[1]), dev::bf16_pack2(v[2], v[3])};
                }
            };
            if (o == 1)
              stage([](float g, float) { return g; });
            else if (o == 2)
              stage([](float, float u) { return u; });
            else
              dev::with_gate(a.act, [&](auto kind) CBD_INLINE { stage([&](float g, float u) { return kind.act(g) * u; }); });
            asm volatile("" ::: "memory");  // a wave's LDS accesses run in order
#pragma unroll
            for (int it = 0; it < 2 * GM; it++) {
              const int row = (64 / CH) * it + lane / CH, ch = lane % CH;
              const u32x4 v = *(const u32x4*)(st + row * 128 + ((ch ^ (row & 7)) << 4));
              put(c, outs[o], lds[o], 64 * n + 32 * wn + row, 32 * GM * wm + 8 * ch, v);
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < L * UNITS; i++) {
          const int n = i / UNITS, h = i % UNITS;
          if constexpr (MB == 4) {
#pragma unroll
            for (int m = 0; m < 2; m++) asm volatile("" : "+a"(acc[2 * h + m][n]));
          }
          const Gates x = ahead[EARLY ? i : 0];
          if (!EARLY && i + 1 < L * UNITS) fetch(c, (i + 1) / UNITS, (i + 1) % UNITS, ahead[0]);
#pragma unroll
          for (int half = 0; half < 2; half++) {
            char* const st = st0 + (SBUF == 2 && half ? 4096 : 0);
            // 16 rows of 64 features, chunk k (4 of them) of row r at k ^ r.
            if ((r >> 4) == half) {
#pragma unroll
              for (int m = 0; m < 2; m++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                  *(f32x4*)(st + (r & 15) * 256 + (((8 * m + 2 * q + hi) ^ (r & 15)) << 4)) =
                      f32x4{acc[2 * h + m][n][4 * q], acc[2 * h + m][n][4 * q + 1], acc[2 * h + m][n][4 * q + 2],
                            acc[2 * h + m][n][4 * q + 3]};
            }
            asm volatile("" ::: "memory");
#pragma unroll
            for (int it = 0; it < 2; it++) {
              const int row = 8 * it + (lane >> 3), ch = lane & 7;
              u32x4 dg, du;
              dev::with_gate(a.act, [&](auto kind) CBD_INLINE {
#pragma unroll
                for (int p = 0; p < 2; p++) {
                  const f32x4 dh = *(const f32x4*)(st + row * 256 + (((2 * ch + p) ^ row) << 4));
                  float vg[4], vu[4];
#pragma unroll
                  for (int j = 0; j < 4; j++) {
                    const uint32_t wg = x.g[2 * half + it][2 * p + (j >> 1)], wu = x.u[2 * half + it][2 * p + (j >> 1)];
                    const float g = __uint_as_float(j & 1 ? wg & 0xffff0000u : wg << 16);
                    const float u = __uint_as_float(j & 1 ? wu & 0xffff0000u : wu << 16);
                    float slope;
                    vu[j] = dh[j] * kind.act(g, &slope);
                    vg[j] = dh[j] * u * slope;
                  }
#pragma unroll
                  for (int j = 0; j < 2; j++) {
                    dg[2 * p + j] = dev::bf16_pack2(vg[2 * j], vg[2 * j + 1]);
                    du[2 * p + j] = dev::bf16_pack2(vu[2 * j], vu[2 * j + 1]);
                  }
                }
              });
              const int at = 64 * n + 32 * wn + 16 * half + row, f = 32 * MB * wm + 64 * h + 8 * ch;
              put(c, c.out, a.ldo, at, f, dg);
              put(c, c.out + a.M, a.ldo, at, f, du);
            }
            asm volatile("" ::: "memory");
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      deep = PAIR && OUT == WHOLE && L == NB;
    }
  };

  Tiles tiles;
  tiles.init(a, BN);
  // Halves in the last round, of 256 rows only: 18432 rows to 2048 outputs (576
  // tiles) 137 us with halves, 146 without at 2048 inputs, 49 / 54 at 512; with
  // 128 x 128 tiles, 10240 rows to 1000 outputs (640), 20.0 / 17.9.
  const int halves = NB == 4 ? (int)gridDim.x : 0;
  int64_t b = blockIdx.x;
  dev::ExpertTile t = tiles.at(a, b, BN, halves);
  if (!t.ok) return;
  Tile c = begin(t);

  // A tile with L of the NB row blocks.
  auto product = [&](auto lc, int KT) CBD_INLINE {
    f32x16 acc[MB][decltype(lc)::value];
    constexpr int L = decltype(lc)::value;
    constexpr int RA = FeedA::READS, RB = FeedB::READS;
    constexpr int Q = MB * L;            // MFMAs of 16 k
    constexpr int R = MB * RA + L * RB;  // fragment reads of 16 k
    // The reads end some MFMAs before the wait that follows them.
    constexpr int RQ = Q >= 8 ? Q - 4 : Q > 1 ? Q - 1 : 1;
    bf16x8 a0[MB], a1[MB], b0[L], b1[L];
    const f32x16 zero = {};
    [[maybe_unused]] Gates ahead[EARLY ? UNITS * L : 1];
    // Between the tile's first loads and the main loop's.
    auto fetch_early = [&]() CBD_INLINE {
      if constexpr (EARLY) {
#pragma unroll
        for (int i = 0; i < UNITS * L; i++) fetch(c, i / UNITS, i % UNITS, ahead[i]);
      }
    };
    auto read_one = [&](int stage, int ks, int r, bf16x8 (&ra)[MB], bf16x8 (&rb)[L]) CBD_INLINE {
      // In the order of use: A block 0, B block 0, the other A, the other B.
      if (r < RA || (r >= RA + RB && r < MB * RA + RB)) {
        const int i = r < RA ? r : r - RB;
        fa.read(smem + stage * FeedA::BYTES, i / RA, ks, i % RA, ra[i / RA]);
      } else {
        const int i = r < RA + RB ? r - RA : r - MB * RA;
        fb.read(smem + BBASE + stage * FeedB::BYTES, i / RB, ks, i % RB, rb[i / RB]);
      }
    };
    if constexpr (DMA) {
      // 16 k: MFMAs on (xa, xb), reading (ya, yb) of the next 16 k and
      // issuing an operand's loads in between.  The order is pinned: a wave
      // issues an instruction every four clocks at most, and an MFMA takes 32.
      auto part = [&](auto firstc, const bf16x8 (&xa)[MB], const bf16x8 (&xb)[L], int stage, int ks,
                      bf16x8 (&ya)[MB], bf16x8 (&yb)[L], auto nc, auto&& load) CBD_INLINE {
        constexpr int LOADS = decltype(nc)::value;
#pragma unroll
        for (int q = 0; q < Q; q++) {
          const int n = q / MB, m = (n & 1) ? MB - 1 - q % MB : q % MB;
          acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[m], xb[n], firstc.value ? zero : acc[m][n], 0, 0, 0);
#pragma unroll
          for (int r = q * R / RQ; r < (q + 1) * R / RQ && r < R; r++) read_one(stage, ks, r, ya, yb);
#pragma unroll
          for (int i = q * LOADS / Q; i < (q + 1) * LOADS / Q; i++) load(i);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      constexpr std::integral_constant<int, 0> none{};
      constexpr std::integral_constant<int, FeedA::N> all_a{};
      constexpr std::integral_constant<int, NS == 2 ? 0 : FeedB::N> all_b{};
      (void)all_b;
      constexpr int STEP = FeedA::N + FeedB::N;  // loads of a step
      // Step 0 has landed: of the tile's first loads, all but these are done.
      constexpr int AHEAD = NS == 2 ? STEP : (NS - 2) * STEP + FeedA::N;
      if (deep)
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(AHEAD + STORES));
      else
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(AHEAD));
      __builtin_amdgcn_s_barrier();
      fetch_early();
#pragma unroll
      for (int r = 0; r < R; r++) read_one(0, 0, r, a0, b0);
      // Loads past the last step fetch zeros (a record count of 0); the next
      // tile's first loads follow them in order.
      //
      // 64 k, step kt in stage S: the first quarter loads the rows of step
      // kt + 1 (step 1's came with the tile's first loads).  Before the last
      // quarter, step kt + 1 has landed and every wave has read the rest of
      // stage S (barrier); the last quarter loads the features of step kt + 2
      // into it.
      //
      // 32 k: the first half loads the rows of step kt + 3; before the second,
      // step kt + 1 has landed (two more steps are on their way) and stage S
      // is read; the second half loads the features of step kt + 4 into it.
      // The last tile's stores are newer than what the first two steps wait
      // for.
      auto iter = [&](int kt, auto sc, auto firstc) CBD_INLINE {
        constexpr int S = decltype(sc)::value;
        constexpr bool FIRST = decltype(firstc)::value;
        if constexpr (NS == 2) {
          part(firstc, a0, b0, S, 1, a1, b1, std::integral_constant<int, FIRST ? 0 : FeedB::N>(),
               [&](int i) { issue_b(1 - S, i); });
          if (!FIRST) fb.advance(kt + 2, KT);
          part(std::false_type(), a1, b1, S, 2, a0, b0, none, [](int) {});
          part(std::false_type(), a0, b0, S, 3, a1, b1, none, [](int) {});
          if (FIRST && deep)
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(STORES));
          else
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
          __builtin_amdgcn_s_barrier();
          part(std::false_type(), a1, b1, 1 - S, 0, a0, b0, all_a, [&](int i) { issue_a(S, i); });
          fa.advance(kt + 3, KT);
        } else {
          part(firstc, a0, b0, S, 1, a1, b1, all_b, [&](int i) { issue_b((S + NS - 1) % NS, i); });
          fb.advance(kt + NS, KT);
          if ((FIRST || kt == 1) && deep)
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((NS - 2) * STEP + STORES));
          else
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((NS - 2) * STEP));
          __builtin_amdgcn_s_barrier();
          part(std::false_type(), a1, b1, (S + 1) % NS, 0, a0, b0, all_a, [&](int i) { issue_a(S, i); });
          fa.advance(kt + NS + 1, KT);
        }
      };
      iter(0, std::integral_constant<int, 0>(), std::true_type());
#pragma unroll 1
      for (int kt = 1; kt < KT; kt += NS) {
        iter(kt, std::integral_constant<int, 1>(), std::false_type());
        if constexpr (NS > 2) {
          if (kt + 1 < KT) iter(kt + 1, std::integral_constant<int, 2>(), std::false_type());
          if (kt + 2 < KT) iter(kt + 2, std::integral_constant<int, 3>(), std::false_type());
        }
        if (kt + NS - 1 < KT) iter(kt + NS - 1, std::integral_constant<int, 0>(), std::false_type());
      }
    } else {
#pragma unroll
      for (int m = 0; m < MB; m++)
#pragma unroll
        for (int n = 0; n < L; n++) acc[m][n] = zero;
      // Everyone has read the stages of the last tile.
      __syncthreads();
      fa.stage(smem);
      fb.stage(smem + BBASE);
      fa.load(fa.K - BK);
      fb.load(fa.K - BK);
      auto iter = [&](int kt, auto sc) CBD_INLINE {
        constexpr int S = decltype(sc)::value;
        // Stage S is filled, and everyone has read stage 1 - S.
        __syncthreads();
        fa.stage(smem + (1 - S) * FeedA::BYTES);
        fb.stage(smem + BBASE + (1 - S) * FeedB::BYTES);
        fa.load(fa.K - (kt + 2) * BK);
        fb.load(fa.K - (kt + 2) * BK);
#pragma unroll
        for (int ks = 0; ks < BK / 16; ks++) {
#pragma unroll
          for (int r = 0; r < R; r++) read_one(S, ks, r, a0, b0);
#pragma unroll
          for (int q = 0; q < Q; q++)
            acc[q % MB][q / MB] =
                __builtin_amdgcn_mfma_f32_32x32x16_bf16(a0[q % MB], b0[q / MB], acc[q % MB][q / MB], 0, 0, 0);
        }
      };
#pragma unroll 1
      for (int kt = 0; kt < KT; kt += 2) {
        iter(kt, std::integral_constant<int, 0>());
        if (kt + 1 < KT) iter(kt + 1, std::integral_constant<int, 1>());
      }
    }
    const Tile done = c;
    if constexpr (GATE == GATE_BWD && !EARLY) fetch(done, 0, 0, ahead[0]);
    if (t.ok) c = begin(t);
    if constexpr (GATE == GATE_NONE)
      finish(done, lc, acc);
    else
      finish_gated(done, lc, acc, ahead);
  };
  // Zeros, where nothing is contracted (added: nothing to do).
  auto blank = [&]() CBD_INLINE {
    // The tile's loads (zeros) land before its stages' next ones.
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    const Tile done = c;
    if (t.ok) c = begin(t);
    deep = false;
    if (OUT == WHOLE_ADD || (OUT == ANY && a.accumulate)) return;
    constexpr int PER = 16 / sizeof(TO), ROWS = THREADS / (FEATS / PER);
    const int tid = fresh_tid(), f = PER * (tid % (FEATS / PER));
#pragma unroll 1
    for (int row = tid / (FEATS / PER); row < BN && row < done.nrows; row += ROWS) {
      TO* o = done.out + row * a.ldo + f;
      if (done.mrows - f >= PER) {
        *(u32x4u*)o = u32x4{0u, 0u, 0u, 0u};
      } else {
#pragma unroll 1
        for (int j = 0; f + j < done.mrows; j++) o[j] = TO(0);
      }
    }
    if constexpr (GATE == GATE_FWD_SAVE || GATE == GATE_BWD) {
      // The other places that the tile's features have.
      const int64_t ld = GATE == GATE_BWD ? a.ldo : a.ldgu;
      TO* const first = GATE == GATE_BWD ? done.out + a.M : (TO*)a.gu + done.n0 * a.ldgu + done.m0;
#pragma unroll 1
      for (int part = 0; part < (GATE == GATE_BWD ? 1 : 2); part++)
#pragma unroll 1
        for (int row = tid / (FEATS / PER); row < BN && row < done.nrows; row += ROWS) {
          TO* o = first + part * (int64_t)a.M + row * ld + f;
#pragma unroll 1
          for (int j = 0; j < PER && f + j < done.mrows; j++) o[j] = TO(0);
        }
    }
  };

  do {
    b += gridDim.x;
    t = tiles.at(a, b, BN, halves);
    const int KT = __builtin_amdgcn_readfirstlane((c.K + BK - 1) / BK);
    if (KT == 0)
      blank();
    else if (c.nrows > 64 * (NB - 1))
      product(std::integral_constant<int, NB>(), KT);
    else if (NB <= 2 || c.nrows <= 64)
      product(std::integral_constant<int, 1>(), KT);
    else if (c.nrows <= 128)
      product(std::integral_constant<int, (NB > 1 ? 2 : 1)>(), KT);
    else
      product(std::integral_constant<int, (NB > 1 ? NB - 1 : 1)>(), KT);
  } while (t.ok);
}

}  // namespace
}  // namespace cbd
