// block_api.cpp -- plans, argument checks and launches of the norms around a block.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <string>

#include "block_internal.h"
#include "cbd_internal.h"
#include "expert_common.h"

namespace {

using cbd::host::Block;
using cbd::host::esize;
using cbd::host::fail;
using cbd::host::guarded;
using cbd::host::share;

cbd_status make_plan(const cbd_block_problem* q, cbd_block_plan_t** out) {
  if (!q || !out) return fail(CBD_ERR_INVALID_ARG, "NULL problem or output");
  *out = nullptr;
  if (q->rows < 0 || q->c < 1) return fail(CBD_ERR_INVALID_ARG, "rows must be >= 0 and c >= 1");
  if (q->dtype != CBD_F32 && q->dtype != CBD_BF16) return fail(CBD_ERR_INVALID_ARG, "unknown dtype");
  if (q->dw_dtype != CBD_F32 && !(q->dw_dtype == CBD_BF16 && q->dtype == CBD_BF16))
    return fail(CBD_ERR_INVALID_ARG, "dw_dtype must be f32, or bf16 with bf16 rows");
  if (!(q->eps >= 0.0) || !std::isfinite((float)q->eps) || !std::isfinite((float)q->scale))
    return fail(CBD_ERR_INVALID_ARG, "eps must be finite and >= 0, scale finite");
  if (q->rows > (int64_t(1) << 40)) return fail(CBD_ERR_UNSUPPORTED, "more than 2^40 rows");
  if (q->c > cbd::kBlockMaxC) return fail(CBD_ERR_UNSUPPORTED, "more than 16384 elements a row");
  cbd_block_plan_s* p = new (std::nothrow) cbd_block_plan_s;
  if (!p) return fail(CBD_ERR_NO_MEMORY, "out of host memory");
  p->prob = *q;
  p->shape = cbd::block_shape(q->c, esize(q->dtype));
  const int threads = cbd::block_threads(p->shape), per = threads / p->shape.lanes;
  const int64_t groups = (q->rows + per - 1) / per;
  // Workgroups that stay.  Forward, as many as the compute units hold at once (8
  // waves a SIMD; half as many: 4096 rows of 4096 in bf16 27 / 30 us, 32768 rows
  // alike).  Backward, as many as have 512 threads with elements a compute unit:
  // twice that have more sums to join (32768 x 4096 in bf16 301 / 324 us and 5.0 /
  // 6.4 for the joining, 512 rows 15 / 21 and 4.0 / 4.7; 65536 x 128 20 / 22 and 4.4
  // / 6.7), and counted with the idle threads of a row's last part there are too few
  // loads on their way (250 MB in bf16, of 1032 335 / 453 us, 264 328 / 445, 2560
  // 302 / 347).  Below 64 threads a row three workgroups fit.
  const int chunks = (int)((q->c * esize(q->dtype) + 15) / 16), most = p->shape.lanes < 64 ? 3 : 1024 / threads;
  const int active = std::min(chunks, p->shape.lanes) * per, wanted = (512 + active / 2) / active;
  p->grid_fwd = std::min<int64_t>(groups, 256 * (2048 / threads));
  p->grid_bwd = std::min<int64_t>(groups, 256 * std::max(1, std::min(wanted, most)));
  // Sums that are held in LDS are of no more than kBlockJoin rows each, with more
  // workgroups than the card has at once; past 4096 of them (2^19 rows, 9 GB at least)
  // of a 4096th of the rows.
  if (!cbd::block_held(p->shape.chunks, esize(q->dtype)))
    p->grid_bwd = std::max(p->grid_bwd, std::min<int64_t>((q->rows + cbd::kBlockJoin - 1) / cbd::kBlockJoin, 4096));
  // A few rows (groups of them) by one workgroup, which then needs no second
  // launch to join its sums with others' (one / many and the joining, us: a row of
  // 4096 9.1 / 12.9, four 13.1 / 13.1, eight 18.2 / 13.2; four groups of four rows
  // of 512 5.6 / 7.1, eight 7.4 / 7.3).
  if (groups <= 4) p->grid_bwd = 1;
  *out = p;
  cbd::set_error("");
  return CBD_OK;
}

uint64_t workspace(const cbd_block_plan_s& p) {
  return ((uint64_t)std::max<int64_t>(p.grid_bwd, 1) * 2 * p.prob.c * sizeof(float) + 255) / 256 * 256;
}

struct Parts {
  cbd_block_params p;
  cbd_block_strides s;
};

// The parameters and strides of a call, or what is wrong with them.
cbd_status read_parts(const cbd_block_problem& q, const void* r, const void* y, const cbd_block_params* params,
                      const cbd_block_strides* st, Parts& o) {
  o.p = {nullptr, nullptr, nullptr, CBD_GATE_NONE, 0};
  if (params) o.p = *params;
  if (o.p.reserved) return fail(CBD_ERR_INVALID_ARG, "the reserved parameter must be zero");
  if (o.p.gate_kind < CBD_GATE_NONE || o.p.gate_kind > CBD_GATE_ROW)
    return fail(CBD_ERR_INVALID_ARG, "unknown gate_kind");
  const bool rows = q.rows > 0;
  if (rows && !r) return fail(CBD_ERR_INVALID_ARG, "NULL r");
  if ((o.p.gate_kind == CBD_GATE_CHANNEL) != (o.p.gate && o.p.gate_kind != CBD_GATE_ROW) ||
      (o.p.gate_kind == CBD_GATE_ROW && rows && !o.p.gate))
    return fail(CBD_ERR_INVALID_ARG, "gate and gate_kind do not go together");
  if (rows && !y && (o.p.w_post || o.p.gate_kind != CBD_GATE_NONE))
    return fail(CBD_ERR_INVALID_ARG, "w_post and gate need y");
  o.s = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
  if (st) o.s = *st;
  for (int64_t* v : {&o.s.r, &o.s.y, &o.s.gate, &o.s.z, &o.s.n, &o.s.dz, &o.s.dn, &o.s.dr, &o.s.dy, &o.s.dgate}) {
    if (!*v) *v = q.c;
    if (*v < q.c) return fail(CBD_ERR_INVALID_ARG, "a row stride is smaller than the row");
    if (*v > (int64_t(1) << 31)) return fail(CBD_ERR_UNSUPPORTED, "a stride is too large");
  }
  return CBD_OK;
}

// What a call touches; `same`: the input that an output may be, exactly.
struct Touch {
  Block b;
  bool out;
  const void* same;
  int64_t same_ld;
};

cbd_status check(const Touch* t, int n) {
  for (int i = 0; i < n; i++)
    if ((uintptr_t)t[i].b.p & (uintptr_t)(t[i].b.es - 1))
      return fail(CBD_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
  for (int i = 0; i < n; i++)
    for (int j = 0; t[i].out && t[i].b.p && j < n; j++) {
      if (j == i || !t[j].b.p) continue;
      const bool itself = !t[j].out && t[i].b.p == t[i].same && t[j].b.p == t[i].same && t[i].b.ld == t[i].same_ld &&
                          t[j].b.ld == t[i].same_ld;
      if (!itself && share(t[i].b, t[j].b)) return fail(CBD_ERR_INVALID_ARG, "an output overlaps another tensor");
    }
  return CBD_OK;
}

cbd_status done(int err) {
  if (err) {
    cbd::set_error(std::string("block norm kernel launch failed: ") + cbd::hip_error_name(err));
    return CBD_ERR_HIP;
  }
  cbd::set_error("");
  return CBD_OK;
}

cbd::BlockArgs arguments(const cbd_block_problem& q, const Parts& o, const void* r, const void* y) {
  cbd::BlockArgs a = {};
  a.r = r;
  a.y = y;
  a.gate = o.p.gate;
  a.gate_rows = o.p.gate_kind == CBD_GATE_ROW;
  a.w_post = o.p.w_post;
  a.w_pre = o.p.w_pre;
  a.ldr = o.s.r;
  a.ldy = o.s.y;
  a.ldgate = o.s.gate;
  a.ldz = o.s.z;
  a.ldn = o.s.n;
  a.lddz = o.s.dz;
  a.lddn = o.s.dn;
  a.lddr = o.s.dr;
  a.lddy = o.s.dy;
  a.lddgate = o.s.dgate;
  a.rows = q.rows;
  a.c = (int32_t)q.c;
  a.eps = (float)q.eps;
  a.scale = (float)q.scale;
  return a;
}

cbd_status forward(const cbd_block_plan_t* plan, const void* r, const void* y, const cbd_block_params* params, void* z,
                   void* n, float* stats, const cbd_block_strides* st, void* stream) {
  if (!plan) return fail(CBD_ERR_INVALID_ARG, "NULL plan");
  const cbd_block_problem& q = plan->prob;
  Parts o;
  const cbd_status bad = read_parts(q, r, y, params, st, o);
  if (bad != CBD_OK) return bad;
  if (q.rows > 0 && ((y != nullptr) != (z != nullptr) || (o.p.w_pre != nullptr) != (n != nullptr)))
    return fail(CBD_ERR_INVALID_ARG, "z goes with y, and n with w_pre");
  const int es = esize(q.dtype);
  const Touch t[] = {
      {{r, q.rows, q.c, o.s.r, 1, 0, es}, false, nullptr, 0},
      {{y, q.rows, q.c, o.s.y, 1, 0, es}, false, nullptr, 0},
      {{o.p.gate, o.p.gate_kind == CBD_GATE_ROW ? q.rows : 1, q.c, o.s.gate, 1, 0, es}, false, nullptr, 0},
      {{o.p.w_post, 1, q.c, q.c, 1, 0, es}, false, nullptr, 0},
      {{o.p.w_pre, 1, q.c, q.c, 1, 0, es}, false, nullptr, 0},
      {{z, q.rows, q.c, o.s.z, 1, 0, es}, true, r, o.s.r},
      {{n, q.rows, q.c, o.s.n, 1, 0, es}, true, y, o.s.y},
      {{stats, q.rows, 2, 2, 1, 0, 4}, true, nullptr, 0},
  };
  const cbd_status over = check(t, 8);
  if (over != CBD_OK) return over;
  if (!q.rows || (!z && !n && !stats)) return done(0);
  cbd::BlockArgs a = arguments(q, o, r, y);
  a.z = z;
  a.n = n;
  a.stats = stats;
  return done(cbd::launch_block_forward(a, plan->shape, q.dtype, plan->grid_fwd, stream));
}

cbd_status bwd(const cbd_block_plan_t* plan, const void* dz, const void* dn, const void* r, const void* y,
               const float* stats, const cbd_block_params* params, const cbd_block_grads* grads,
               const cbd_block_strides* st, void* ws, uint64_t ws_bytes, void* stream) {
  if (!plan || !grads) return fail(CBD_ERR_INVALID_ARG, "NULL plan or gradients");
  const cbd_block_problem& q = plan->prob;
  Parts o;
  const cbd_status bad = read_parts(q, r, y, params, st, o);
  if (bad != CBD_OK) return bad;
  const cbd_block_grads& g = *grads;
  const bool row_gate = o.p.gate_kind == CBD_GATE_ROW;
  if (q.rows > 0 && !stats && (o.p.w_post || o.p.w_pre)) return fail(CBD_ERR_INVALID_ARG, "NULL stats");
  if (q.rows > 0 && !y && g.dy) return fail(CBD_ERR_INVALID_ARG, "dy needs y");
  if ((g.dw_post && !o.p.w_post) || (g.dgate && o.p.gate_kind == CBD_GATE_NONE) || (g.dw_pre && !o.p.w_pre))
    return fail(CBD_ERR_INVALID_ARG, "the gradient of a parameter that is not given");
  if (dn && !o.p.w_pre) return fail(CBD_ERR_INVALID_ARG, "dn needs w_pre");
  void* const dgate_row = row_gate ? g.dgate : nullptr;
  const bool vectors = g.dw_post || g.dw_pre || (g.dgate && !row_gate);
  const uint64_t need = workspace(*plan);
  if (vectors && (!ws || ws_bytes < need))
    return fail(CBD_ERR_INVALID_ARG, "no workspace, or one smaller than cbd_block_workspace_size");
  if (vectors && (uintptr_t)ws & 255u) return fail(CBD_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  const int es = esize(q.dtype), ws_es = esize(q.dw_dtype);
  const Touch t[] = {
      {{r, q.rows, q.c, o.s.r, 1, 0, es}, false, nullptr, 0},
      {{y, q.rows, q.c, o.s.y, 1, 0, es}, false, nullptr, 0},
      {{dz, q.rows, q.c, o.s.dz, 1, 0, es}, false, nullptr, 0},
      {{dn, q.rows, q.c, o.s.dn, 1, 0, es}, false, nullptr, 0},
      {{o.p.gate, row_gate ? q.rows : 1, q.c, o.s.gate, 1, 0, es}, false, nullptr, 0},
      {{o.p.w_post, 1, q.c, q.c, 1, 0, es}, false, nullptr, 0},
      {{o.p.w_pre, 1, q.c, q.c, 1, 0, es}, false, nullptr, 0},
      {{stats, q.rows, 2, 2, 1, 0, 4}, false, nullptr, 0},
      {{g.dr, q.rows, q.c, o.s.dr, 1, 0, es}, true, dz, o.s.dz},
      {{g.dy, q.rows, q.c, o.s.dy, 1, 0, es}, true, dn, o.s.dn},
      {{dgate_row, q.rows, q.c, o.s.dgate, 1, 0, es}, true, nullptr, 0},
      {{g.dw_post, 1, q.c, q.c, 1, 0, ws_es}, true, nullptr, 0},
      {{row_gate ? nullptr : g.dgate, 1, q.c, q.c, 1, 0, ws_es}, true, nullptr, 0},
      {{g.dw_pre, 1, q.c, q.c, 1, 0, ws_es}, true, nullptr, 0},
      {{vectors ? ws : nullptr, 1, (int64_t)need, (int64_t)need, 1, 0, 1}, true, nullptr, 0},
  };
  const cbd_status over = check(t, 15);
  if (over != CBD_OK) return over;
  if (!vectors && (!q.rows || (!g.dr && !g.dy && !dgate_row))) return done(0);
  cbd::BlockFinish f = {};
  f.partial = (const float*)ws;
  f.gate = row_gate ? nullptr : o.p.gate;
  f.w_post = o.p.w_post;
  f.dw_post = g.dw_post;
  f.dgate = row_gate ? nullptr : g.dgate;
  f.dw_pre = g.dw_pre;
  f.n = q.rows ? (int32_t)plan->grid_bwd : 0;
  f.c = (int32_t)q.c;
  f.dtype = q.dtype;
  f.dw_dtype = q.dw_dtype;
  int err = 0;
  if (q.rows) {
    cbd::BlockArgs a = arguments(q, o, r, y);
    a.dz = dz;
    a.dn = dn;
    if (!dn) a.w_pre = nullptr;
    a.dr = g.dr;
    a.dy = g.dy;
    a.dgate = dgate_row;
    a.stats = const_cast<float*>(stats);
    a.partial = vectors ? (float*)ws : nullptr;
    a.finish = f;
    err = cbd::launch_block_bwd(a, plan->shape, q.dtype, plan->grid_bwd, stream);
  }
  if (!err && vectors && f.n != 1) err = cbd::launch_block_finish(f, stream);
  return done(err);
}

}  // namespace

extern "C" cbd_status cbd_block_plan(const cbd_block_problem* problem, cbd_block_plan_t** out_plan) {
  return guarded([&] { return make_plan(problem, out_plan); });
}

extern "C" void cbd_block_plan_destroy(cbd_block_plan_t* plan) { delete plan; }

extern "C" cbd_status cbd_block_workspace_size(const cbd_block_plan_t* plan, uint64_t* bytes) {
  return guarded([&]() -> cbd_status {
    if (!plan || !bytes) return fail(CBD_ERR_INVALID_ARG, "NULL plan or output");
    *bytes = workspace(*plan);
    return CBD_OK;
  });
}

extern "C" cbd_status cbd_block_forward(const cbd_block_plan_t* plan, const void* r, const void* y,
                                        const cbd_block_params* params, void* z, void* n, float* stats,
                                        const cbd_block_strides* strides, void* stream) {
  return guarded([&] { return forward(plan, r, y, params, z, n, stats, strides, stream); });
}

extern "C" cbd_status cbd_block_bwd(const cbd_block_plan_t* plan, const void* dz, const void* dn, const void* r,
                                    const void* y, const float* stats, const cbd_block_params* params,
                                    const cbd_block_grads* grads, const cbd_block_strides* strides, void* workspace,
                                    uint64_t workspace_bytes, void* stream) {
  return guarded([&] {
    return bwd(plan, dz, dn, r, y, stats, params, grads, strides, workspace, workspace_bytes, stream);
  });
}
