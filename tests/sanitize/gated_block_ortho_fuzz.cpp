// Host fuzz of the entry points of the gated experts, the norms around a block
// and the orthogonalised updates for a sanitizer build: random problems, strides
// and addresses.  The launchers are replaced by checks of what they are handed:
// every call returns a status, nothing is launched on an error, what is launched
// keeps to the limits that the kernels rely on, and everything that the products
// of an orthogonalisation read and write lies inside its workspace, what is read
// having been written before.  Built with -fsanitize=address,undefined by
// tests/test_host_sanitizers_more.py.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <string>
#include <vector>

#include "block_internal.h"
#include "cbd_internal.h"
#include "gated_internal.h"
#include "ortho_internal.h"

static long launches, checked;
static int broken;
static void expect(bool ok, const char* what) {
  checked++;
  if (ok || broken) return;
  std::fprintf(stderr, "broken: %s\n", what);
  broken = 1;
}

namespace cbd {
void set_error(const std::string&) {}
const char* hip_error_name(int) { return "error"; }
int launch_expert_generic(const ExpertArgs&, const ExpertLaunch&, void*) { return 0; }
int launch_expert_mfma(const ExpertArgs&, const ExpertLaunch&, void*) { return 0; }
int launch_expert_stream(const ExpertArgs&, const ExpertLaunch&, void*) { return 0; }

// ---- gated experts

static int gated(const GatedArgs& a, const ExpertLaunch& l, int mode, int kernel) {
  launches++;
  const int64_t es = l.dtype == CBD_F32 ? 4 : 2, lim = int64_t(1) << 31;
  const bool pair = mode != GATE_BWD;
  expect(l.kernel == kernel && l.grid >= 1 && l.grid < (int64_t(1) << 24), "grid");
  expect(l.form == EXPERT_AK || l.form == EXPERT_AM, "form");
  expect(a.E >= 1 && a.T >= 1 && a.M >= 1 && a.K >= 1 && a.tiles_m == (a.M + l.bm - 1) / l.bm, "sizes");
  expect(a.ldb >= a.K && a.lda >= 1 && a.ldo >= (pair ? 1 : 2) * a.M, "strides");
  expect(a.ldb * 256 * es < lim && a.ldo * 256 * es < lim, "rows of a tile pass 32-bit offsets");
  expect(mode == GATE_FWD || (a.gu && a.ldgu >= 2 * a.M && a.ldgu * 256 * es < lim), "gu");
  expect(((uintptr_t)a.out & (es - 1)) == 0 && ((uintptr_t)a.ends & (a.ends64 ? 7 : 3)) == 0, "alignment");
  const int64_t feats = pair ? 2 * a.M : a.M;
  const int64_t slice = l.form == EXPERT_AK ? (feats - 1) * a.lda + a.K : (int64_t)(a.K - 1) * a.lda + feats;
  expect(slice * es < lim && a.a_expert >= slice, "an expert's weights");
  expect(!pair || a.up == (l.form == EXPERT_AK ? a.M * a.lda : a.M), "the second projection");
  if (l.dma) {
    expect((((uintptr_t)a.a | (uintptr_t)a.b) & 15) == 0 && a.lda % 8 == 0 && a.ldb % 8 == 0, "16-byte rows");
    expect(a.K % 8 == 0 && (!pair || a.up % 8 == 0) && a.lda * 256 * es < lim, "16-byte steps");
  }
  if (a.whole_out)
    expect(((uintptr_t)a.out & 15) == 0 && a.ldo * es % 16 == 0 && a.M * es % 16 == 0 &&
               (mode == GATE_FWD || (((uintptr_t)a.gu & 15) == 0 && a.ldgu * es % 16 == 0)),
           "whole results");
  const int wide = pair ? 2 * l.bm : l.bm;
  if (kernel == CBD_EXPERT_KERNEL_MFMA) {
    expect(l.dtype == CBD_BF16 && wide == l.bn && (l.bn == 128 || (l.bn == 256 && l.dma && a.whole_out)), "tile");
    const int64_t tiles = (int64_t)a.tiles_m * (a.T / l.bn + std::min(a.E + 1, a.T));
    expect(tiles <= INT32_MAX && (l.grid == tiles || l.grid == (l.bn == 256 ? 256 : 512)), "workgroups that stay");
  } else if (kernel == CBD_EXPERT_KERNEL_GENERIC) {
    expect(wide == l.bn && (l.bn == 128 || l.bn == 64), "tile");
  } else {
    expect(l.dtype == CBD_BF16 && pair && l.bn == 32 && wide == (l.form == EXPERT_AK ? 32 : 128) && a.lda * 256 * es < lim,
           "stream");
  }
  return 0;
}
int launch_gated_generic(const GatedArgs& a, const ExpertLaunch& l, int mode, void*) {
  return gated(a, l, mode, CBD_EXPERT_KERNEL_GENERIC);
}
int launch_gated_mfma(const GatedArgs& a, const ExpertLaunch& l, int mode, void*) {
  return gated(a, l, mode, CBD_EXPERT_KERNEL_MFMA);
}
int launch_gated_stream(const GatedArgs& a, const ExpertLaunch& l, int mode, void*) {
  return gated(a, l, mode, CBD_EXPERT_KERNEL_STREAM);
}

// ---- norms around a block

static uint64_t workspace;  // of the plan in use
static void block(const BlockArgs& a, BlockShape s, int dtype, int64_t grid) {
  launches++;
  const int es = dtype == CBD_F32 ? 4 : 2;
  expect(a.c >= 1 && (int64_t)s.lanes * s.chunks * 16 >= (int64_t)a.c * es, "the shape covers a row");
  expect(s.lanes >= 8 && s.lanes <= 1024 && (s.lanes & (s.lanes - 1)) == 0, "lanes");
  expect(s.chunks == 1 || (s.lanes == 1024 && (s.chunks == 2 || (s.chunks == 4 && es == 4))), "an instance of the kernel");
  expect(grid >= 1 && grid <= 256 * 16 && a.rows >= 1 && a.r, "grid");
  expect(!(a.w_post || a.gate) || a.y, "parts");
}
int launch_block_forward(const BlockArgs& a, BlockShape s, int dtype, int64_t grid, void*) {
  block(a, s, dtype, grid);
  expect((a.z != nullptr) == (a.y != nullptr) && (a.n != nullptr) == (a.w_pre != nullptr), "outputs");
  return 0;
}
int launch_block_bwd(const BlockArgs& a, BlockShape s, int dtype, int64_t grid, void*) {
  block(a, s, dtype, grid);
  expect(!a.partial || (uint64_t)grid * 2 * a.c * 4 <= workspace, "partial sums");
  expect(!(a.w_post || a.w_pre) || a.stats, "stats");
  expect(a.finish.c == a.c && a.finish.n == grid, "finish");
  return 0;
}
int launch_block_finish(const BlockFinish& a, void*) {
  launches++;
  expect(a.partial && a.c >= 1 && a.n != 1 && (uint64_t)a.n * 2 * a.c * 4 <= workspace, "finish");
  return 0;
}

// ---- orthogonalised updates

static const char *ws_begin, *ws_end;
static int64_t count;  // matrices
static const float* sliced;  // sums that wait to be joined
static int64_t done;   // of them, by the launches of the product so far
// Extents of halves that have been written, as (begin, rows, halves of a row that hold values, ld, mat).
struct Area {
  const uint16_t* p;
  int64_t rows, used, ld, mat;
};
static std::vector<Area> written;
static void inside(const void* p, int64_t halves_per_matrix, int64_t mat, const char* what) {
  const char* b = (const char*)p;
  expect(b >= ws_begin && b + 2 * ((count - 1) * mat + halves_per_matrix) <= ws_end && ((uintptr_t)b & 15) == 0 && mat % 8 == 0,
         what);
}
static void wrote(const uint16_t* p, int64_t rows, int64_t used, int64_t ld, int64_t mat) {
  expect(used <= ld && rows * ld <= mat, "a matrix's rows and pitch");
  inside(p, (rows - 1) * ld + used, mat, "a store outside the workspace");
  for (Area& w : written)
    if (w.p == p) {
      w = {p, rows, used, ld, mat};
      return;
    }
  written.push_back({p, rows, used, ld, mat});
}
// The first `need` rows and all the contracted side have to be there; whole tiles are loaded.
static void read(const uint16_t* p, int64_t need, int64_t tile_rows, int64_t used, int64_t ld, int64_t mat) {
  inside(p, (tile_rows - 1) * ld + used, mat, "a load outside the workspace");
  bool found = false;
  for (const Area& w : written)
    if (w.p == p) found = w.rows >= need && w.used >= used && w.ld == ld && w.mat == mat;
  expect(found, "an operand that was not written");
}
int launch_ortho_norm(const OrthoSplit& a, int64_t matrices, void*) {
  launches++;
  count = matrices;
  written.clear();
  done = 0;
  expect((const char*)a.partial >= ws_begin && (const char*)(a.partial + matrices * kOrthoParts) <= ws_end, "norms");
  return 0;
}
int launch_ortho_split(const OrthoSplit& a, int64_t matrices, void*) {
  launches++;
  const int64_t r = (a.rows + 63) / 64 * 64, c = (a.cols + 63) / 64 * 64;
  expect((a.rows + 63) / 64 <= 65535 && matrices <= 65535, "grid");
  wrote(a.x, r, 2 * c, a.ldx, a.x_mat);
  wrote(a.xt, c, 2 * r, a.ldxt, a.xt_mat);
  return 0;
}
int launch_ortho_product(const OrthoArgs& share, int stage, int tile, int64_t matrices, void*) {
  launches++;
  expect(matrices >= 1 && done + matrices <= count, "matrices of a product");
  // As if one launch did them all.
  OrthoArgs a = share;
  a.p -= done * a.p_mat;
  a.q -= done * a.q_mat;
  if (a.c) a.c -= done * a.c_mat;
  if (a.ct) a.ct -= done * a.ct_mat;
  done = done + matrices == count ? 0 : done + matrices;
  const bool sym = stage == ORTHO_SQUARE || stage == ORTHO_POLY || stage == ORTHO_SLICE;
  expect(tile == 64 || tile == 128 || tile == 256, "tile");
  expect((int64_t)a.tiles_m * a.tiles_n * matrices < (int64_t(1) << 24), "grid");
  expect(a.tiles_m == (a.rows + tile - 1) / tile && a.tiles_n == (a.cols + tile - 1) / tile, "tiles");
  expect(a.runs >= 1 && 64 * a.runs <= a.ldp && 64 * a.runs <= a.ldq, "runs");
  expect((int64_t)tile * a.ldp * 2 < INT32_MAX && (int64_t)tile * a.ldq * 2 < INT32_MAX, "32-bit offsets");
  read(a.p, a.rows, (int64_t)tile * a.tiles_m, 64 * a.runs, a.ldp, a.p_mat);
  read(a.q, a.cols, (int64_t)tile * a.tiles_n, 64 * a.runs, a.ldq, a.q_mat);
  const int64_t m = (int64_t)tile * a.tiles_m, n = (int64_t)tile * a.tiles_n;
  if (stage == ORTHO_SLICE) {
    const char* const b = (const char*)a.sums;
    const int64_t tiles = a.tiles_m * (a.tiles_m + 1) / 2 * count;
    expect(tile == 64 && matrices == count && tiles * a.slices <= 256, "slices in one round");
    expect(a.slices >= 2 && a.slice * (a.slices - 1) < a.runs && a.runs <= a.slice * a.slices, "every run in one slice");
    expect(b >= ws_begin && ((uintptr_t)b & 15) == 0 && b + tiles * a.slices * 64 * 64 * 4 <= ws_end, "sums");
    for (const Area& w : written)
      expect(b + tiles * a.slices * 64 * 64 * 4 <= (const char*)w.p || (const char*)(w.p + count * w.mat) <= b, "sums over a matrix");
    sliced = a.sums;
    return 0;
  }
  if (stage == ORTHO_POLY) inside(a.p, (m - 1) * a.ldp + 2 * n, a.p_mat, "A outside the workspace");
  if (stage == ORTHO_LAST) {
    expect(a.out && a.out_row >= (a.flip ? a.rows : a.cols), "output");
    return 0;
  }
  for (const uint16_t* in : {a.p, a.q}) expect(a.c != in && a.ct != in, "a product over its own operand");
  wrote(a.c, m, 2 * n, a.ldc, a.c_mat);
  wrote(a.ct, n, 2 * m, a.ldct, a.ct_mat);
  expect(!sym || (a.c == a.ct && a.ldc == a.ldct && a.rows == a.cols), "symmetric");
  return 0;
}
int launch_ortho_join(const OrthoArgs& a, int64_t matrices, void*) {
  launches++;
  expect(a.sums && a.sums == sliced && matrices == count && a.tiles_m == (a.rows + 63) / 64 && a.tiles_n == a.tiles_m, "joining");
  expect(a.c == a.ct && a.ldc == a.ldct && a.rows == a.cols && a.c != a.p, "symmetric");
  sliced = nullptr;
  wrote(a.c, 64 * a.tiles_m, 2 * 64 * a.tiles_n, a.ldc, a.c_mat);
  return 0;
}
}  // namespace cbd

template <typename R>
static int64_t pick(R& rng, std::initializer_list<int64_t> v) {
  return *(v.begin() + rng() % v.size());
}
static bool status(cbd_status r) {
  return r == CBD_OK || r == CBD_ERR_INVALID_ARG || r == CBD_ERR_UNSUPPORTED;
}

static void gated(std::mt19937_64& rng, long iters) {
  auto uni = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  for (long it = 0; it < iters; it++) {
    cbd_expert_problem p = {};
    p.tokens = rng() % 8 ? uni(0, 70000) : pick(rng, {0, 1, 1 << 20, 1 << 30});
    p.experts = rng() % 8 ? uni(1, 130) : pick(rng, {1, 65536});
    p.c = rng() % 8 ? uni(1, 5000) : pick(rng, {1, 8, 1 << 20});
    p.k = rng() % 8 ? uni(1, 5000) : pick(rng, {1, 2, 16, 1 << 20});
    if (rng() % 2) p.c = (p.c + 15) / 16 * 16, p.k = (p.k + 15) / 16 * 16;
    p.w_layout = (int32_t)uni(0, 1);
    p.dtype = p.dw_dtype = (int32_t)uni(0, 1);
    p.ends_bits = (int32_t)pick(rng, {32, 64});
    cbd_expert_options o = {(int32_t)uni(-1, 2), {0, 0, 0}};
    cbd_expert_plan_t* plan = nullptr;
    if (cbd_expert_plan(&p, rng() % 3 ? nullptr : &o, &plan) != CBD_OK) continue;
    uint64_t at[5];
    for (int i = 0; i < 5; i++) at[i] = ((uint64_t)(i + 1) << 56) + 16 * (rng() % 64);
    if (rng() % 4 == 0) at[rng() % 5] += pick(rng, {1, 2, 4, 8});
    if (rng() % 10 == 0) at[rng() % 5] = at[rng() % 5] + 2 * (rng() % 9000);
    if (rng() % 40 == 0) at[rng() % 5] = 0;
    auto ptr = [&](int i) { return (void*)(uintptr_t)at[i]; };
    for (int bwd = 0; bwd < 2; bwd++) {
      cbd_expert_info_t info;
      expect(cbd_expert_gated_info(plan, bwd, &info) == (bwd || p.k % 2 == 0 ? CBD_OK : CBD_ERR_INVALID_ARG), "info");
      const int64_t m = bwd ? p.c : p.k / 2, in = bwd ? p.k : p.c;
      const int64_t wr = p.w_layout == CBD_EXPERT_EKC ? p.k : p.c, ww = p.w_layout == CBD_EXPERT_EKC ? p.c : p.k;
      cbd_gated_strides s = {};
      if (rng() % 2) s.in_row = in + pick(rng, {-1, 0, 1, 8, 64, 1 << 22, (int64_t)1 << 40});
      if (rng() % 2) s.h_row = m + pick(rng, {-1, 0, 1, 8, 64, 1 << 22});
      if (rng() % 2) s.gu_row = 2 * m + pick(rng, {-1, 0, 1, 8, 64, 1 << 22});
      if (rng() % 2) s.dgu_row = 2 * m + pick(rng, {-1, 0, 1, 8, 64, 1 << 22});
      if (rng() % 2) s.w_row = ww + pick(rng, {-1, 0, 1, 8, 64, 1 << 20});
      if (rng() % 2) s.w_expert = (wr - 1) * (s.w_row ? s.w_row : ww) + ww + pick(rng, {-1, 0, 1, 8, 64, (int64_t)1 << 41});
      const cbd_gated_strides* sp = rng() % 2 ? &s : nullptr;
      const int32_t act = (int32_t)(rng() % 20 ? uni(0, 2) : pick(rng, {-1, 3}));
      const long before = launches;
      const cbd_status r =
          bwd ? cbd_expert_gated_bwd(plan, ptr(0), ptr(1), ptr(3), ptr(2), ptr(4), act, sp, nullptr)
              : cbd_expert_gated_forward(plan, ptr(0), ptr(1), ptr(2), ptr(3), rng() % 2 ? ptr(4) : nullptr, act, sp, nullptr);
      expect(r == CBD_OK ? launches <= before + 1 : launches == before, "a launch after an error");
      expect(status(r), "status");
      expect(r != CBD_OK || (act >= 0 && act <= 2), "an unknown activation");
    }
    cbd_expert_plan_destroy(plan);
  }
}

static void blocks(std::mt19937_64& rng, long iters) {
  auto uni = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  for (long it = 0; it < iters; it++) {
    cbd_block_problem q = {};
    q.rows = rng() % 8 ? uni(0, 100000) : pick(rng, {-1, 0, 1, 5, (int64_t)1 << 40, ((int64_t)1 << 40) + 1});
    q.c = rng() % 8 ? uni(1, 16384) : pick(rng, {0, 1, 7, 16384, 16385});
    q.dtype = (int32_t)(rng() % 30 ? uni(0, 1) : 4);
    q.dw_dtype = (int32_t)uni(0, 1);
    q.eps = rng() % 30 ? 1e-6 : -1.0;
    q.scale = 0.5;
    cbd_block_plan_t* plan = nullptr;
    const cbd_status st = cbd_block_plan(&q, &plan);
    expect((st == CBD_OK) == (plan != nullptr) && status(st), "a status and its plan");
    if (!plan) continue;
    expect(cbd_block_workspace_size(plan, &cbd::workspace) == CBD_OK && cbd::workspace % 256 == 0, "workspace size");
    void* at[16];
    for (int i = 0; i < 16; i++) at[i] = (void*)(((uint64_t)(i + 1) << 58 >> 2) + 256 * (rng() % 64));
    if (rng() % 6 == 0) at[rng() % 16] = (char*)at[rng() % 16] + pick(rng, {0, 1, 2, 4, 4096});
    if (rng() % 4 == 0) at[rng() % 16] = nullptr;
    cbd_block_strides s = {};
    int64_t* const all[] = {&s.r, &s.y, &s.gate, &s.z, &s.n, &s.dz, &s.dn, &s.dr, &s.dy, &s.dgate};
    for (int64_t* v : all)
      if (rng() % 4 == 0) *v = q.c + pick(rng, {0, 0, 1, 8, 64, -1, (int64_t)1 << 32});
    const cbd_block_strides* sp = rng() % 2 ? &s : nullptr;
    cbd_block_params w = {rng() % 3 ? at[2] : nullptr, rng() % 3 ? at[3] : nullptr, rng() % 3 ? at[4] : nullptr, 0, 0};
    w.gate_kind = (int32_t)(rng() % 10 ? (w.gate ? uni(1, 2) : 0) : uni(-1, 3));
    void* const y = rng() % 5 ? at[1] : nullptr;
    if (!y && rng() % 3) w = {nullptr, nullptr, w.w_pre, 0, 0};
    long before = launches;
    cbd_status r = cbd_block_forward(plan, at[0], y, &w, y && rng() % 20 ? (rng() % 4 ? at[5] : at[0]) : nullptr,
                                     w.w_pre && rng() % 20 ? (rng() % 4 ? at[6] : y) : nullptr,
                                     rng() % 2 ? (float*)at[7] : nullptr, sp, nullptr);
    expect(status(r) && (r == CBD_OK ? launches <= before + 1 : launches == before), "forward");
    cbd_block_grads g = {rng() % 4 ? at[10] : nullptr, y && rng() % 4 ? at[11] : nullptr, w.w_post && rng() % 4 ? at[12] : nullptr,
                         w.gate && rng() % 4 ? at[13] : nullptr, w.w_pre && rng() % 4 ? at[14] : nullptr};
    before = launches;
    r = cbd_block_bwd(plan, rng() % 5 ? at[8] : nullptr, w.w_pre && rng() % 5 ? at[9] : nullptr, at[0], y, (float*)at[7], &w, &g,
                      sp, at[15], rng() % 10 ? cbd::workspace : cbd::workspace - 1, nullptr);
    expect(status(r) && (r == CBD_OK ? launches <= before + 2 : launches == before), "backward");
    cbd_block_plan_destroy(plan);
  }
}

static void ortho(std::mt19937_64& rng, long iters) {
  auto uni = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  for (long it = 0; it < iters; it++) {
    cbd_ortho_problem q = {};
    q.matrices = rng() % 8 ? uni(0, 40) : pick(rng, {-1, 0, 1, 1000, 65535, 65536});
    q.rows = rng() % 4 ? uni(1, 5000) : pick(rng, {0, 1, 31, 32, 33, 63, 64, 65, 128, 65536, 65537});
    q.cols = rng() % 4 ? uni(1, 5000) : pick(rng, {0, 1, 31, 32, 33, 63, 64, 65, 128, 65536, 65537});
    q.dtype = (int32_t)(rng() % 30 ? uni(0, 1) : 2);
    q.steps = (int32_t)(rng() % 30 ? uni(1, 8) : pick(rng, {0, 64, 65}));
    q.eps = rng() % 30 ? 1e-7 : 0.0;
    q.scale = 1.0;
    std::vector<double> co;
    if (rng() % 3 == 0) {
      for (int i = 0; i < 3 * std::max(q.steps, 0); i++) co.push_back((double)(int64_t)(rng() % 2001) / 100.0 - 10.0);
      q.coefficients = co.data();
      if (q.steps < 1) q.coefficients = nullptr;
    }
    cbd_ortho_plan_t* plan = nullptr;
    const cbd_status st = cbd_ortho_plan(&q, &plan);
    expect((st == CBD_OK) == (plan != nullptr) && status(st), "a status and its plan");
    if (!plan) continue;
    uint64_t size = 0;
    cbd_ortho_info_t info;
    expect(cbd_ortho_workspace_size(plan, &size) == CBD_OK && cbd_ortho_plan_info(plan, &info) == CBD_OK, "sizes");
    uint64_t at[3] = {(uint64_t)1 << 60, (uint64_t)2 << 60, (uint64_t)3 << 60};
    if (rng() % 6 == 0) at[rng() % 3] += pick(rng, {1, 2, 4, 256});
    if (rng() % 10 == 0) at[1] = at[0] + 4 * (rng() % 3);
    if (rng() % 30 == 0) at[rng() % 3] = 0;
    cbd_ortho_strides s = {};
    if (rng() % 3 == 0) s.in_row = q.cols + pick(rng, {-1, 0, 1, 64, (int64_t)1 << 32});
    if (rng() % 3 == 0) s.out_row = q.cols + pick(rng, {-1, 0, 1, 64, (int64_t)1 << 32});
    if (rng() % 3 == 0) s.in_matrix = q.rows * (s.in_row ? s.in_row : q.cols) + pick(rng, {-1000000, 0, 5, (int64_t)1 << 41});
    cbd::ws_begin = (const char*)at[2];
    cbd::ws_end = cbd::ws_begin + size;
    const long before = launches;
    const cbd_status r = cbd_orthogonalize(plan, (void*)at[0], (void*)at[1], rng() % 2 ? &s : nullptr, (void*)at[2],
                                           rng() % 10 ? size : size - 1, nullptr);
    expect(status(r) && (r == CBD_OK ? launches - before == info.launches : launches == before), "orthogonalize");
    cbd_ortho_plan_destroy(plan);
  }
}

int main(int argc, char** argv) {
  const long iters = argc > 1 ? std::atol(argv[1]) : 10000;
  std::mt19937_64 rng(argc > 2 ? std::atoll(argv[2]) : 1);
  gated(rng, iters);
  const long a = launches;
  blocks(rng, iters);
  const long b = launches;
  ortho(rng, iters / 4);
  std::printf("launches: %ld gated, %ld blocks, %ld updates; checks: %ld\n", a, b - a, launches - b, checked);
  return broken || a < iters / 10 || b - a < iters / 10 || launches - b < iters / 10;
}
