// The tile enumeration of the expert products (csrc/expert_device.h), run on
// the host: 64 contexts stand for a wave's lanes and swap at every operation
// that crosses lanes.  Every row of every feature tile, every feature of a row
// of slices that start early, and every tile of a weight gradient has to have
// exactly one workgroup.
//
//   expert_tiles SEED COUNT
#include <setjmp.h>
#include <ucontext.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <random>
#include <vector>

struct Index {
  unsigned x;
};
static Index threadIdx;

namespace wave {
constexpr int LANES = 64;
static ucontext_t lanes[LANES], home;  // to start a lane; then jumps, which cost no system call
static jmp_buf at[LANES];
static bool started[LANES];
static int slot[2][LANES], parity[LANES];
static std::vector<char> stacks(LANES * 64 * 1024);
static std::function<void(int)> body;
static bool done[LANES];

[[noreturn]] static void go(int n) {
  threadIdx.x = (unsigned)n;
  if (started[n]) _longjmp(at[n], 1);
  started[n] = true;
  setcontext(&lanes[n]);
  std::abort();
}
__attribute__((noinline)) static void yield() {
  const int l = (int)threadIdx.x;
  if (!_setjmp(at[l])) go((l + 1) % LANES);
}
// Every lane's v: lanes run in turn, so all have written when this one is back.
static const int* exchange(int v) {
  const int l = (int)threadIdx.x, p = parity[l] ^= 1;
  slot[p][l] = v;
  yield();
  return slot[p];
}
static void entry() {
  const int l = (int)threadIdx.x;
  body(l);
  done[l] = true;
  if (l < LANES - 1) go(l + 1);
  setcontext(&home);
}
// Runs f on 64 lanes; all have to cross lanes equally often.
static void run(std::function<void(int)> f) {
  body = std::move(f);
  for (int l = 0; l < LANES; l++) {
    getcontext(&lanes[l]);
    lanes[l].uc_stack = {};
    lanes[l].uc_stack.ss_sp = stacks.data() + l * 64 * 1024;
    lanes[l].uc_stack.ss_size = 64 * 1024;
    lanes[l].uc_link = nullptr;
    makecontext(&lanes[l], entry, 0);
    started[l] = done[l] = false;
  }
  threadIdx.x = 0;
  started[0] = true;
  swapcontext(&home, &lanes[0]);
  for (bool d : done)
    if (!d) {
      std::fprintf(stderr, "lanes diverged\n");
      std::exit(1);
    }
}

static int dpp(int old, int v, int ctrl, int rows, int banks, bool) {
  const int* s = exchange(v);
  const int l = (int)threadIdx.x, row = l / 16;
  int from = -1;
  if (ctrl >= 0x111 && ctrl <= 0x11f)
    from = l % 16 >= (ctrl & 15) ? l - (ctrl & 15) : -1;  // row_shr
  else if (ctrl == 0x142)
    from = row > 0 ? 16 * row - 1 : -1;                   // row_bcast:15
  else if (ctrl == 0x143)
    from = row > 1 ? 31 : -1;                             // row_bcast:31
  else if (ctrl == 0x138)
    from = l - 1;                                         // wave_shr:1
  else
    std::abort();
  if (banks != 15) std::abort();
  return from < 0 || !(rows >> row & 1) ? old : s[from];
}
static int readlane(int v, int l) { return exchange(v)[l]; }
static unsigned long long ballot(bool p) {
  const int* s = exchange(p);
  unsigned long long m = 0;
  for (int l = 0; l < LANES; l++) m |= (unsigned long long)(s[l] != 0) << l;
  return m;
}
}  // namespace wave

#define __device__
#define __ballot(p) wave::ballot(p)
#define __builtin_amdgcn_update_dpp wave::dpp
#define __builtin_amdgcn_readlane wave::readlane
#define __builtin_amdgcn_readfirstlane(v) wave::readlane(v, 0)
#include "expert_device.h"

using cbd::ExpertArgs;
using cbd::dev::ExpertTile;

static int fail(const char* what, const ExpertArgs& a, int bn, int g) {
  std::fprintf(stderr, "%s: T=%d E=%d tiles_m=%d tiles_n=%d bn=%d g=%d\n", what, a.T, a.E, a.tiles_m, a.tiles_n, bn, g);
  return 1;
}

// The rows of expert e by the definition; e == E: those past the last one's.
static std::vector<std::pair<int, int>> spans(const std::vector<int>& ends, int T) {
  std::vector<std::pair<int, int>> s;
  int at = 0;
  for (int v : ends) {
    const int hi = std::max(at, std::min(std::max(v, 0), T));
    s.push_back({at, hi});
    at = hi;
  }
  s.push_back({at, T});
  return s;
}

static bool same(const ExpertTile& x, const ExpertTile& y) {
  return x.e == y.e && x.begin == y.begin && x.end == y.end && x.m_tile == y.m_tile && x.n_tile == y.n_tile;
}

// Tiles of all workgroups; g: workgroups that stay (0: one tile each).
template <typename Tiles>
static bool tiles_of(const ExpertArgs& a, int bn, int g, int64_t grid, std::vector<ExpertTile>& out) {
  bool agree = true;
  for (int64_t b = 0; b < grid; b++) {
    const size_t start = out.size();  // lane 0 is ahead of the others
    wave::run([&](int lane) {
      Tiles t = {};
      t.init(a, bn);
      size_t n = start;
      for (int64_t i = b;; i += g) {
        const ExpertTile r = t.at(a, i, bn, g);
        if (r.ok && lane == 0) out.push_back(r);
        if (r.ok) agree = agree && n < out.size() && same(out[n], r), n++;
        if (!r.ok || !g) break;
      }
      agree = agree && n == out.size();
    });
  }
  return agree;
}

static int rows(ExpertArgs a, const std::vector<int>& ends, int bn, int cap) {
  a.ends = ends.data();
  // The grid of a launch: an upper bound of the tiles, or workgroups that stay.
  const int64_t bound = (int64_t)a.tiles_m * (a.T / bn + std::min(a.E + 1, a.T));
  const int64_t grid = cap ? std::min<int64_t>(bound, cap) : bound;
  const int g = cap ? (int)grid : 0;
  std::vector<ExpertTile> tiles;
  if (!tiles_of<cbd::dev::RowTiles>(a, bn, g, grid, tiles)) return fail("lanes disagree", a, bn, g);
  const auto s = spans(ends, a.T);
  std::vector<uint8_t> owned((size_t)a.T * a.tiles_m);
  for (const ExpertTile& t : tiles) {
    if (t.e < 0 || t.e > a.E || t.m_tile < 0 || t.m_tile >= a.tiles_m) return fail("no such tile", a, bn, g);
    if (t.begin < s[t.e].first || t.end > s[t.e].second || t.begin >= t.end || t.end - t.begin > bn)
      return fail("rows of another expert, none or too many", a, bn, g);
    for (int r = t.begin; r < t.end; r++)
      if (owned[(size_t)r * a.tiles_m + t.m_tile]++) return fail("a row with two workgroups", a, bn, g);
  }
  if (std::count(owned.begin(), owned.end(), 1) != (long)owned.size()) return fail("a row without a workgroup", a, bn, g);
  return 0;
}

static int weights(ExpertArgs a, const std::vector<int>& ends, int cap) {
  a.ends = ends.data();
  const int64_t total = (int64_t)a.tiles_m * a.tiles_n * a.E, grid = cap ? std::min<int64_t>(total, cap) : total;
  std::vector<ExpertTile> tiles;
  if (!tiles_of<cbd::dev::WeightTiles>(a, 0, cap ? (int)grid : 0, grid, tiles)) return fail("lanes disagree", a, 0, cap);
  const auto s = spans(ends, a.T);
  std::vector<uint8_t> owned((size_t)total);
  for (const ExpertTile& t : tiles) {
    if (t.begin != s[t.e].first || t.end != s[t.e].second) return fail("not the expert's rows", a, 0, cap);
    if (owned[((size_t)t.e * a.tiles_m + t.m_tile) * a.tiles_n + t.n_tile]++) return fail("a tile twice", a, 0, cap);
  }
  if ((int64_t)tiles.size() != total) return fail("a tile missing", a, 0, cap);
  return 0;
}

static int slices(int bm, int M) {
  std::vector<uint8_t> owned(M);
  for (int i = 0; i * bm < M; i++) {
    const cbd::dev::FeatureSlice s = cbd::dev::feature_slice(i, bm, M);
    if (s.m0 < 0 || s.skip < 0 || (M >= bm && s.m0 + bm > M))
      return std::fprintf(stderr, "slice %d of %d features leaves the row\n", i, M), 1;
    for (int f = s.m0 + s.skip; f < std::min(s.m0 + bm, M); f++)
      if (owned[f]++) return std::fprintf(stderr, "feature %d of %d has two workgroups\n", f, M), 1;
  }
  if (std::count(owned.begin(), owned.end(), 1) != M) return std::fprintf(stderr, "a feature of %d is left out\n", M), 1;
  return 0;
}

int main(int argc, char** argv) {
  std::mt19937 rng(argc > 1 ? std::atoi(argv[1]) : 1);
  const int count = argc > 2 ? std::atoi(argv[2]) : 20;
  auto uni = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int m = 1; m < 1000; m++)
    if (slices(128, m)) return 1;
  ExpertArgs a = {};
  // Tiles left for the last round of 256 workgroups that stay: at and around a
  // half of them, of one expert and of two that end inside a tile, with and
  // without rows past the last one's.
  for (int left : {0, 1, 126, 127, 128, 129, 130, 254, 255})
    for (int rounds : {0, 1, 2})
      for (int tail : {0, 1, 300}) {
        const int n = 256 * rounds + left - (tail + 255) / 256;
        if (n < 1) continue;
        a.tiles_m = 1;
        a.T = 256 * n + tail;
        const int part = 256 * n - uni(0, 255);
        a.E = 1;
        if (rows(a, {256 * n}, 256, 256)) return 1;
        a.E = 2;
        if (rows(a, {256 * (n / 2) + uni(0, 255), part}, 256, 256)) return 1;
      }
  for (int i = 0; i < count; i++) {
    a.E = i % 3 == 0 ? uni(65, 200) : uni(1, 64);
    a.T = uni(1, i % 4 ? 30000 : 300);
    a.tiles_m = uni(1, 9);
    a.tiles_n = uni(1, 9);
    std::vector<int> ends(a.E);
    for (int& v : ends) v = uni(0, a.T);
    std::sort(ends.begin(), ends.end());
    for (int j = 0; j < a.E; j++)
      if (uni(0, 3) == 0) ends[j] = j ? ends[j - 1] : 0;  // no rows
    if (i % 5 == 4) std::shuffle(ends.begin(), ends.end(), rng);
    if (i % 7 == 6) ends[uni(0, a.E - 1)] = uni(0, 1) ? INT_MAX : INT_MIN;
    for (int bn : {64, 128, 256})
      if (rows(a, ends, bn, bn == 256 ? 256 : 512)) return 1;
    if (a.T < 3000)
      for (int bn : {32, 64, 128})
        if (rows(a, ends, bn, 0)) return 1;
    if (weights(a, ends, 256) || weights(a, ends, 512)) return 1;
  }
  std::printf("cases: %d\n", count);
  return 0;
}
