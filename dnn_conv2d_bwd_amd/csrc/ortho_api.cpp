// ortho_api.cpp -- plans, argument checks and launches of the orthogonalised updates.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <string>

#include "cbd_internal.h"
#include "expert_common.h"
#include "ortho_internal.h"

namespace {

using cbd::host::Block;
using cbd::host::esize;
using cbd::host::fail;
using cbd::host::guarded;
using cbd::host::share;

constexpr int kTop = 14;  // stored values stay below 2^14 times what rounding adds (halves end at 2^16)

int64_t up_to(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// The exponent that brings a bound to at most 2^kTop; false if there is none.
bool exponent(double bound, int& e) {
  if (!(bound >= std::ldexp(1.0, -20) && bound <= std::ldexp(1.0, 20))) return false;
  e = kTop - (int)std::ceil(std::log2(bound));
  return true;
}

struct Tile {
  int t;
  double one, two;
};
// Measured, in us a run of 32 of the contracted side, with one workgroup a compute
// unit and with two (256 x 256: one after the other, at the rate that the card's
// power allows when all are busy).  So the last product of a step takes (64 / 128 /
// 256 in us) 11 / 14 / 33 for 16 matrices of 256 x 512, 70 / 51 / 116 for one of
// 2048 x 2048, 483 / 354 / 303 for one of 4096 x 4096 and 83 / 53 / 74 for four of
// 1024 x 2048.
constexpr Tile kTiles[] = {{256, 2.4, 4.8}, {128, 0.58, 1.38}, {64, 0.22, 0.5}};
constexpr double kLaunch = 4.0;  // us of another launch
constexpr double kJoin = 6.0;    // and of one that joins slices' sums

double time_of(const Tile& c, int64_t tiles) {
  const int64_t rest = tiles % 512;
  return (double)(tiles / 512) * c.two + (rest > 256 ? c.two : rest ? c.one : 0.0);
}

// How n matrices with tiles(t) tiles of t x t each and `runs` runs are computed:
// in the tiles that take the least time over all their rounds on the card, or the
// first ones in larger and the rest in smaller tiles, where that leaves fewer
// units idle in the end (A of 8 matrices of 2048 x 4096, 36 tiles of 256 each: 7 in
// one round of those and the last in tiles of 128 387 us, all in tiles of 128
// 404).
template <typename F>
void share_out(int64_t n, int64_t runs, F&& tiles, cbd::OrthoShare (&out)[2]) {
  auto best = [&](int64_t count, double& least) {
    int at = 0;
    least = 0.0;
    for (int i = 0; i < 3; i++) {
      const double time = time_of(kTiles[i], count * tiles(kTiles[i].t));
      if (i == 0 || time < least) {
        at = i;
        least = time;
      }
    }
    return at;
  };
  double least = 0.0;
  out[0] = {kTiles[best(n, least)].t, n};
  out[1] = {64, 0};
  for (int i = 0; i < 2; i++) {
    // Whole rounds of the larger tiles.
    const int64_t per = tiles(kTiles[i].t), round = i == 0 ? 256 : 512;
    for (int64_t r = 1; r <= 64 && r * round / per < n; r++) {
      const int64_t k = r * round / per;
      if (!k) continue;
      double rest = 0.0;
      const int at = best(n - k, rest);
      const double time = time_of(kTiles[i], k * per) + rest + kLaunch / (double)runs;
      if (at > i && time < least) {
        least = time;
        out[0] = {kTiles[i].t, k};
        out[1] = {kTiles[at].t, n - k};
      }
    }
  }
}

cbd_status make_plan(const cbd_ortho_problem* q, cbd_ortho_plan_t** out) {
  if (!q || !out) return fail(CBD_ERR_INVALID_ARG, "NULL problem or output");
  *out = nullptr;
  if (q->matrices < 0 || q->rows < 1 || q->cols < 1)
    return fail(CBD_ERR_INVALID_ARG, "matrices must be >= 0, rows and cols >= 1");
  if (q->dtype != CBD_F32 && q->dtype != CBD_BF16) return fail(CBD_ERR_INVALID_ARG, "unknown dtype");
  if (q->steps < 1 || q->steps > 64) return fail(CBD_ERR_INVALID_ARG, "steps must be 1 to 64");
  if (!(q->eps > 0.0) || !std::isfinite(q->eps) || !std::isfinite((float)q->scale))
    return fail(CBD_ERR_INVALID_ARG, "eps must be finite and > 0, scale finite");
  if (q->matrices > 65535 || q->rows > 65536 || q->cols > 65536)
    return fail(CBD_ERR_UNSUPPORTED, "more than 65535 matrices, or sides above 65536");
  std::unique_ptr<cbd_ortho_plan_s> p(new cbd_ortho_plan_s);
  p->prob = *q;
  p->prob.coefficients = nullptr;
  // Bounds of the singular values, of A and of B in each step.
  double top = 1.0;
  for (int k = 0; k <= q->steps; k++) {
    int e = 0;
    if (!exponent(top, e)) return fail(CBD_ERR_UNSUPPORTED, "the steps let singular values grow or shrink too far");
    p->ex.push_back(e);
    if (k == q->steps) break;
    const double usual[3] = {3.4445, -4.7750, 2.0315};
    const double* c = q->coefficients ? q->coefficients + 3 * k : usual;
    for (int i = 0; i < 3; i++) {
      if (!std::isfinite(c[i])) return fail(CBD_ERR_INVALID_ARG, "a coefficient is not finite");
      p->coefficients.push_back(c[i]);
    }
    double most_b = 0.0, most_x = 0.0;
    for (int i = 0; i <= 512; i++) {
      const double x = top * i / 512, b = std::fabs(c[0] + x * x * (c[1] + x * x * c[2]));
      most_b = std::max(most_b, b);
      most_x = std::max(most_x, b * x);
    }
    int ea = 0, eb = 0;
    if (!exponent(top * top, ea) || !exponent(most_b, eb))
      return fail(CBD_ERR_UNSUPPORTED, "the steps let singular values grow or shrink too far");
    p->ea.push_back(ea);
    p->eb.push_back(eb);
    top = most_x;
  }
  p->s = std::min(q->rows, q->cols);
  p->l = std::max(q->rows, q->cols);
  const int64_t n = std::max<int64_t>(q->matrices, 1);
  const int64_t runs = (p->s + 31) / 32;
  auto sym = [&](int64_t t) {
    const int64_t m = (p->s + t - 1) / t;
    return m * (m + 1) / 2;
  };
  auto step = [&](int64_t t) { return ((p->s + t - 1) / t) * ((p->l + t - 1) / t); };
  share_out(n, runs, sym, p->sym);
  share_out(n, runs, step, p->step);
  // A's sums in slices of its contracted side, of 8 runs at least, where its tiles
  // leave most of the card idle and take longer than a launch that joins them (5
  // steps in us, whole / in slices: 256 x 4096, 16 of them, 232 / 138; 64 x 16384
  // 591 / 126; 8 matrices of 64 x 4096 220 / 125; 768 x 2304, 3 slices, 230 / 202;
  // 4 of 256 x 1536 159 / 149).
  p->slices = 1;
  if (p->sym[0].tile == 64 && !p->sym[1].count) {
    const int64_t all = (p->l + 31) / 32, most = std::min(256 / (n * sym(64)), all / 8);
    if (most > 1 && (double)(all - (all + most - 1) / most) * kTiles[2].one > kJoin) {
      p->slice = (all + most - 1) / most;
      p->slices = (all + p->slice - 1) / p->slice;
    }
  }
  int64_t pad = 64;
  for (const auto* shares : {p->sym, p->step})
    for (int i = 0; i < 2; i++) {
      if (!shares[i].count) continue;
      pad = std::max<int64_t>(pad, shares[i].tile);
      if (shares[i].count * std::max(step(shares[i].tile), sym(shares[i].tile)) > cbd::host::kMaxGrid)
        return fail(CBD_ERR_UNSUPPORTED, "too many tiles for one launch");
    }
  // Tiles of 256 take 1.14 times as long where lo is scaled, which makes them sum hi
  // lo and lo hi, then hi hi (5 steps of 8 matrices of 4096 x 2048 7.26 ms, 6.37).  So
  // bf16 updates with such tiles go without: their values have 22 bits down to 2^-17
  // of the bounds above, not to 2^-28, and are off by 2^-39 of them at most, where
  // the results have 8 bits.
  p->lo_up = q->dtype == CBD_BF16 && pad == 256 ? 1.f : 2048.f;
  p->sp = up_to(p->s, pad);
  p->lp = up_to(p->l, pad);
  *out = p.release();
  cbd::set_error("");
  return CBD_OK;
}

// Halves of a matrix in each of the workspace's arrays, and the whole.
struct Layout {
  int64_t x, a;               // halves of X (either direction) and of A or B
  uint64_t parts, sums, bytes;
  explicit Layout(const cbd_ortho_plan_s& p) {
    const uint64_t n = (uint64_t)p.prob.matrices;
    x = 2 * p.sp * p.lp;
    a = 2 * p.sp * p.sp;
    parts = (n * cbd::kOrthoParts * sizeof(double) + 255) / 256 * 256;
    const uint64_t side = (uint64_t)(p.s + 63) / 64, blocks = n * (side * (side + 1) / 2) * (uint64_t)p.slices;
    sums = p.slices > 1 ? blocks * 64 * 64 * sizeof(float) : 0;
    bytes = parts + sums + n * 2 * (3 * (uint64_t)x + 2 * (uint64_t)a) + 256;
  }
};

cbd_status run(const cbd_ortho_plan_t* plan, const void* in, void* out, const cbd_ortho_strides* st, void* ws,
               uint64_t ws_bytes, void* stream) {
  if (!plan) return fail(CBD_ERR_INVALID_ARG, "NULL plan");
  const cbd_ortho_problem& q = plan->prob;
  if (!q.matrices) {
    cbd::set_error("");
    return CBD_OK;
  }
  if (!in || !out || !ws) return fail(CBD_ERR_INVALID_ARG, "NULL tensor or workspace");
  cbd_ortho_strides s = {0, 0, 0, 0};
  if (st) s = *st;
  if (!s.in_row) s.in_row = q.cols;
  if (!s.out_row) s.out_row = q.cols;
  if (s.in_row < q.cols || s.out_row < q.cols) return fail(CBD_ERR_INVALID_ARG, "a row stride is smaller than the row");
  if (s.in_row > (int64_t(1) << 31) || s.out_row > (int64_t(1) << 31))
    return fail(CBD_ERR_UNSUPPORTED, "a stride is too large");
  const int64_t in_span = (q.rows - 1) * s.in_row + q.cols, out_span = (q.rows - 1) * s.out_row + q.cols;
  if (!s.in_matrix) s.in_matrix = in_span;
  if (!s.out_matrix) s.out_matrix = out_span;
  if (s.in_matrix < in_span || s.out_matrix < out_span)
    return fail(CBD_ERR_INVALID_ARG, "a matrix stride is smaller than the matrix");
  if (s.in_matrix > (int64_t(1) << 40) || s.out_matrix > (int64_t(1) << 40))
    return fail(CBD_ERR_UNSUPPORTED, "a stride is too large");
  const Layout lay(*plan);
  if (ws_bytes < lay.bytes) return fail(CBD_ERR_INVALID_ARG, "workspace smaller than cbd_ortho_workspace_size");
  if ((uintptr_t)ws & 255u) return fail(CBD_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  const int es = esize(q.dtype);
  if (((uintptr_t)in | (uintptr_t)out) & (uintptr_t)(es - 1))
    return fail(CBD_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
  const Block bi = {in, q.rows, q.cols, s.in_row, q.matrices, s.in_matrix, es};
  const Block bo = {out, q.rows, q.cols, s.out_row, q.matrices, s.out_matrix, es};
  const Block bw = {ws, 1, (int64_t)lay.bytes, (int64_t)lay.bytes, 1, 0, 1};
  const bool itself = in == out && s.in_row == s.out_row && s.in_matrix == s.out_matrix;
  if ((!itself && share(bi, bo)) || share(bi, bw) || share(bo, bw))
    return fail(CBD_ERR_INVALID_ARG, "the output or the workspace overlaps another tensor");

  const bool tall = q.rows > q.cols;
  const int64_t n = q.matrices;
  double* const partial = (double*)ws;
  float* const sums = (float*)((char*)ws + lay.parts);
  uint16_t* const x = (uint16_t*)((char*)sums + lay.sums);  // rows: the smaller side
  uint16_t* xt = x + n * lay.x;                            // rows: the larger one
  uint16_t* xt_next = xt + n * lay.x;
  uint16_t* const sq = xt_next + n * lay.x;                // A
  uint16_t* const poly = sq + n * lay.a;                   // B
  const int32_t ldx = (int32_t)(2 * plan->lp), ldxt = (int32_t)(2 * plan->sp);

  cbd::OrthoSplit f = {};
  f.in = in;
  f.in_row = s.in_row;
  f.in_mat = s.in_matrix;
  f.rows = (int32_t)q.rows;
  f.cols = (int32_t)q.cols;
  f.dtype = q.dtype;
  f.partial = partial;
  f.eps = q.eps;
  f.up = std::ldexp(1.0, plan->ex[0]);
  f.lo_up = plan->lo_up;
  f.x = tall ? xt : x;
  f.ldx = tall ? ldxt : ldx;
  f.xt = tall ? x : xt;
  f.ldxt = tall ? ldx : ldxt;
  f.x_mat = f.xt_mat = lay.x;
  int err = cbd::launch_ortho_norm(f, n, stream);
  if (!err) err = cbd::launch_ortho_split(f, n, stream);

  auto tiles = [](int64_t v, int t) { return (int32_t)((v + t - 1) / t); };
  // A product of all matrices, share by share.
  auto product = [&](const cbd::OrthoArgs& all, int stage, const cbd::OrthoShare (&shares)[2]) {
    int64_t first = 0;
    for (const cbd::OrthoShare& h : shares) {
      if (!h.count || err) continue;
      cbd::OrthoArgs a = all;
      a.lo_up = plan->lo_up;
      a.lo_down = 1.f / plan->lo_up;
      a.p += first * a.p_mat;
      a.q += first * a.q_mat;
      if (a.c) a.c += first * a.c_mat;
      if (a.ct) a.ct += first * a.ct_mat;
      if (a.out) a.out = (char*)a.out + first * a.out_mat * es;
      a.tiles_m = tiles(a.rows, h.tile);
      a.tiles_n = tiles(a.cols, h.tile);
      err = cbd::launch_ortho_product(a, stage, h.tile, h.count, stream);
      first += h.count;
    }
  };
  for (int k = 0; k < q.steps && !err; k++) {
    const double* c = &plan->coefficients[3 * k];
    const int ex = plan->ex[k], ea = plan->ea[k], eb = plan->eb[k];
    cbd::OrthoArgs a = {};
    a.p = a.q = x;
    a.p_mat = a.q_mat = lay.x;
    a.ldp = a.ldq = ldx;
    a.runs = tiles(plan->l, 32);
    a.rows = a.cols = (int32_t)plan->s;
    a.c = a.ct = sq;
    a.c_mat = a.ct_mat = lay.a;
    a.ldc = a.ldct = ldxt;
    a.mul = (float)std::ldexp(1.0, ea - 2 * ex);
    if (plan->slices > 1) {
      a.sums = sums;
      a.slices = (int32_t)plan->slices;
      a.slice = (int32_t)plan->slice;
      const float mul = a.mul;
      a.mul = 1.f;  // with the joining
      product(a, cbd::ORTHO_SLICE, plan->sym);
      a.mul = mul;
      a.tiles_m = a.tiles_n = tiles(plan->s, 64);
      a.lo_up = plan->lo_up;
      if (!err) err = cbd::launch_ortho_join(a, n, stream);
    } else {
      product(a, cbd::ORTHO_SQUARE, plan->sym);
    }

    a.p = a.q = sq;
    a.p_mat = a.q_mat = lay.a;
    a.ldp = a.ldq = ldxt;
    a.runs = tiles(plan->s, 32);
    a.c = a.ct = poly;
    a.mul = (float)std::ldexp(c[2], eb - 2 * ea);
    a.p_mul = (float)std::ldexp(c[1], eb - ea);
    a.diag = (float)std::ldexp(c[0], eb);
    product(a, cbd::ORTHO_POLY, plan->sym);

    const bool last = k == q.steps - 1;
    a = {};
    a.p = poly;
    a.p_mat = lay.a;
    a.ldp = ldxt;
    a.q = xt;
    a.q_mat = lay.x;
    a.ldq = ldxt;
    a.runs = tiles(plan->s, 32);
    a.rows = (int32_t)plan->s;
    a.cols = (int32_t)plan->l;
    if (last) {
      a.mul = (float)std::ldexp(1.0, -eb - ex);
      a.scale = (float)q.scale;
      a.out = out;
      a.out_row = s.out_row;
      a.out_mat = s.out_matrix;
      a.out_dtype = q.dtype;
      a.flip = tall;
    } else {
      a.mul = (float)std::ldexp(1.0, plan->ex[k + 1] - eb - ex);
      a.c = x;
      a.c_mat = lay.x;
      a.ldc = ldx;
      a.ct = xt_next;
      a.ct_mat = lay.x;
      a.ldct = ldxt;
    }
    product(a, last ? cbd::ORTHO_LAST : cbd::ORTHO_STEP, plan->step);
    std::swap(xt, xt_next);
  }
  if (err) {
    cbd::set_error(std::string("orthogonalising kernel launch failed: ") + cbd::hip_error_name(err));
    return CBD_ERR_HIP;
  }
  cbd::set_error("");
  return CBD_OK;
}

}  // namespace

extern "C" cbd_status cbd_ortho_plan(const cbd_ortho_problem* problem, cbd_ortho_plan_t** out_plan) {
  return guarded([&] { return make_plan(problem, out_plan); });
}

extern "C" void cbd_ortho_plan_destroy(cbd_ortho_plan_t* plan) { delete plan; }

extern "C" cbd_status cbd_ortho_plan_info(const cbd_ortho_plan_t* plan, cbd_ortho_info_t* out) {
  return guarded([&]() -> cbd_status {
    if (!plan || !out) return fail(CBD_ERR_INVALID_ARG, "NULL plan or output");
    const int sym = plan->sym[1].count ? 2 : 1, step = plan->step[1].count ? 2 : 1;
    out->tile_symmetric = plan->sym[0].tile;
    out->tile_step = plan->step[0].tile;
    out->tile_symmetric_rest = plan->sym[1].count ? plan->sym[1].tile : 0;
    out->tile_step_rest = plan->step[1].count ? plan->step[1].tile : 0;
    out->launches = plan->prob.matrices ? 2 + plan->prob.steps * (2 * sym + step + (plan->slices > 1)) : 0;
    out->slices = (int32_t)plan->slices;
    out->flops = plan->prob.matrices * plan->prob.steps * plan->s * plan->s * (3 * plan->l + plan->s);
    cbd::set_error("");
    return CBD_OK;
  });
}

extern "C" cbd_status cbd_ortho_workspace_size(const cbd_ortho_plan_t* plan, uint64_t* bytes) {
  return guarded([&]() -> cbd_status {
    if (!plan || !bytes) return fail(CBD_ERR_INVALID_ARG, "NULL plan or output");
    *bytes = Layout(*plan).bytes;
    return CBD_OK;
  });
}

extern "C" cbd_status cbd_orthogonalize(const cbd_ortho_plan_t* plan, const void* in, void* out,
                                        const cbd_ortho_strides* strides, void* workspace, uint64_t workspace_bytes,
                                        void* stream) {
  return guarded([&] { return run(plan, in, out, strides, workspace, workspace_bytes, stream); });
}
