// expert_device.h -- which rows a workgroup of an expert product owns.  Only
// integers and wave operations, so that a host program can run it too: kernels
// include cbd_device.h first.
#pragma once
#include "cbd_tile.h"
#include "expert_internal.h"

// Inlined always: a kernel's by-value arguments would otherwise be copied to
// memory to be passed by reference.
#define CBD_INLINE __attribute__((always_inline))

namespace cbd {
namespace dev {

// Inclusive scans over the 64 lanes of a wave (values >= 0, so 0 is the
// identity of both): shifts within rows of 16 lanes, then the last lane of
// each row broadcast into the next ones.
__device__ inline int wave_scan_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return v;
}
__device__ inline int wave_scan_max(int v) {
  auto mx = [](int a, int b) { return a > b ? a : b; };
  v = mx(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
  v = mx(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = mx(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = mx(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = mx(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
  v = mx(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
  return v;
}

// ends[i] clamped to [0, T].
CBD_INLINE __device__ inline int clamped_end(const void* ends, int ends64, int i, int T) {
  if (ends64) {
    const int64_t v = ((const int64_t*)ends)[i];
    return v < 0 ? 0 : v > T ? T : (int)v;
  }
  const int v = ((const int32_t*)ends)[i];
  return v < 0 ? 0 : v > T ? T : v;
}

// A value that is the same in every lane, in scalar registers.
CBD_INLINE __device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
CBD_INLINE __device__ inline uint64_t uniform(uint64_t v) {
  return (uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)(uint32_t)v);
}

struct ExpertTile {
  int e;           // expert; E for the rows past the last expert's
  int begin, end;  // AK, AM: the tile's rows; DW: the expert's
  int m_tile, n_tile;
  bool ok;         // false: no such tile (the grid is an upper bound)
};

// One chunk of 64 experts: this lane's row range [lo, hi).  last: the end of
// the chunk before on entry, of this one on exit.
CBD_INLINE __device__ inline void expert_chunk(const ExpertArgs& a, int base, int& last, int& lo, int& hi) {
  const int i = base + (int)(threadIdx.x & 63);
  hi = wave_scan_max(i < a.E ? clamped_end(a.ends, a.ends64, i, a.T) : 0);
  hi = hi > last ? hi : last;
  // The previous lane's hi: wave_shr:1 (lane 0 keeps the last chunk's).
  lo = __builtin_amdgcn_update_dpp(last, hi, 0x138, 0xf, 0xf, false);
  last = __builtin_amdgcn_readlane(hi, 63);
}

// Logical tile of hardware workgroup b: XCD x (b % 8) gets tiles 32 x .. 32 x
// + 31 of every 256, and its share of what is left, so neighbouring tiles meet
// in one L2 while the XCDs' loads stay alike however the experts' sizes vary.
// (Taking the tiles in descending order of their rows instead evens the
// workgroups' loads out better, but reads the weights twice: 256 rows an
// expert 160 -> 177 us.)
CBD_INLINE __device__ inline int spread_tile(int b, int tiles) {
  const int full = tiles & ~255;
  if (b < full) return (b & ~255) + ((b & 7) << 5) + ((b & 255) >> 3);
  return full + logical_tile(b - full, tiles - full, tiles - full >= 64 ? 1 : 0);
}

// Row tiles (of bn rows) of an AK / AM product.  Every wave scans ends itself,
// 64 experts a step, so no barrier is needed; up to 64 experts stay in
// registers.  The tiles of an expert are consecutive, in groups of 8 feature
// tiles by all row tiles; neighbouring workgroups of one XCD then share both
// operands' panels.  Rows past the last expert's come last.
struct RowTiles {
  int lo, hi, n, sum;  // of this lane's expert: rows, row tiles; row tiles of all up to it
  int total, last;     // row tiles of the experts; the last one's end
  int64_t tiles;

  CBD_INLINE __device__ void init(const ExpertArgs& a, int bn) {
    last = total = 0;
    for (int base = 0; base < a.E; base += 64) {
      expert_chunk(a, base, last, lo, hi);
      n = (hi - lo + bn - 1) / bn;
      sum = wave_scan_sum(n);
      total += __builtin_amdgcn_readlane(sum, 63);
    }
    tiles = (int64_t)(total + (a.T - last + bn - 1) / bn) * a.tiles_m;
  }
  // Cuts r's rows down to those of row tile n_tile, or (half 0, 1; -1: all) to
  // a half of it.  A second half may have none.
  CBD_INLINE __device__ static void cut(ExpertTile& r, int bn, int half) {
    r.begin += r.n_tile * bn + (half == 1 ? bn / 2 : 0);
    const int most = half < 0 ? bn : bn / 2;
    r.ok = r.begin < r.end;
    if (r.end - r.begin > most) r.end = r.begin + most;
  }
  // Tile of hardware workgroup b.  g > 0: of workgroups that take b, b + g, ...
  // (g a multiple of 256, or as many as there are tiles); where the last
  // round's tiles are at most g / 2, each is taken as two halves of its rows.
  CBD_INLINE __device__ ExpertTile at(const ExpertArgs& a, int64_t b, int bn, int g = 0) {
    ExpertTile r;
    int half = -1;
    const int64_t whole = g > 0 ? (int)tiles / g * g : tiles;  // fewer than 2^31: the caller checks
    const int left = (int)(tiles - whole);
    if (b >= whole && 2 * left <= g) {
      const int p = b - whole < 2 * left ? logical_tile((int)(b - whole), 2 * left, 1) : 2 * left;
      half = p & 1;
      b = whole + (p >> 1);
    }
    r.ok = b < tiles;
    r.e = a.E;
    r.begin = last;
    r.end = a.T;
    r.m_tile = r.n_tile = 0;
    if (!r.ok) return r;
    const int t = half < 0 ? spread_tile((int)b, (int)tiles) : (int)b;
    if (t >= (int64_t)total * a.tiles_m) {
      const int local = t - total * a.tiles_m;
      r.n_tile = uniform(local / a.tiles_m);
      r.m_tile = uniform(local - r.n_tile * a.tiles_m);
      cut(r, bn, half);
      return r;
    }
    int before = 0, end = 0;  // row tiles and rows before the chunk
    for (int base = 0; base < a.E; base += 64) {
      if (a.E > 64) {
        expert_chunk(a, base, end, lo, hi);
        n = (hi - lo + bn - 1) / bn;
        sum = wave_scan_sum(n);
      }
      const unsigned long long hit = __ballot((int64_t)(before + sum) * a.tiles_m > t);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        const int k = __builtin_amdgcn_readlane(n, l);
        const int first = before + __builtin_amdgcn_readlane(sum, l) - k;
        r.e = base + l;
        r.begin = __builtin_amdgcn_readlane(lo, l);
        r.end = __builtin_amdgcn_readlane(hi, l);
        const int local = t - first * a.tiles_m;
        const int grp = local / (8 * k);
        const int gm = a.tiles_m - 8 * grp < 8 ? a.tiles_m - 8 * grp : 8;
        const int in = local - grp * 8 * k;
        const int row = in / gm;
        r.n_tile = uniform(row);
        r.m_tile = uniform(8 * grp + in - row * gm);
        cut(r, bn, half);
        return r;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
    }
    return r;
  }
};

// Rows of expert e (a DW workgroup knows its expert).
CBD_INLINE __device__ inline void expert_rows(const ExpertArgs& a, int e, int& begin, int& end) {
  int v = 0;
  for (int i = threadIdx.x & 63; i < e; i += 64) {
    const int x = clamped_end(a.ends, a.ends64, i, a.T);
    v = x > v ? x : v;
  }
  begin = __builtin_amdgcn_readlane(wave_scan_max(v), 63);
  const int x = __builtin_amdgcn_readfirstlane(clamped_end(a.ends, a.ends64, e, a.T));
  end = x > begin ? x : begin;
}

// Features of slice i of M by a kernel that loads slices of bm features whole:
// the last one starts early, where there are as many, so that it ends with the
// row; its first `skip` features are the slice's before, which stores them.
struct FeatureSlice {
  int m0, skip;
};
CBD_INLINE __device__ inline FeatureSlice feature_slice(int i, int bm, int M) {
  const int own = i * bm, m0 = own + bm > M && M >= bm ? M - bm : own;
  return {m0, own - m0};
}

// Tiles of a DW product: groups of 8 feature tiles by all tiles of the other
// side, as above.
struct WeightTiles {
  int lo, hi;  // rows of up to 64 experts
  int tiles;

  CBD_INLINE __device__ void init(const ExpertArgs& a, int) {
    tiles = a.tiles_m * a.tiles_n * a.E;
    int last = 0;
    if (a.E <= 64) expert_chunk(a, 0, last, lo, hi);
  }
  CBD_INLINE __device__ ExpertTile at(const ExpertArgs& a, int64_t b, int, int) const {
    ExpertTile r;
    r.ok = b < tiles;
    r.e = r.begin = r.end = r.m_tile = r.n_tile = 0;
    if (!r.ok) return r;
    const int t = spread_tile((int)b, tiles);
    const int per = a.tiles_m * a.tiles_n;
    r.e = uniform(t / per);
    const int local = t - r.e * per;
    const int g = local / (8 * a.tiles_n);
    const int gm = a.tiles_m - 8 * g < 8 ? a.tiles_m - 8 * g : 8;
    const int in = local - g * 8 * a.tiles_n;
    const int row = in / gm;
    r.n_tile = uniform(row);
    r.m_tile = uniform(8 * g + in - row * gm);
    if (a.E <= 64) {
      r.begin = __builtin_amdgcn_readlane(lo, r.e);
      r.end = __builtin_amdgcn_readlane(hi, r.e);
    } else {
      expert_rows(a, r.e, r.begin, r.end);
    }
    return r;
  }
};

}  // namespace dev
}  // namespace cbd
