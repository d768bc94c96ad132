// expert_api.cpp -- plans, argument checks and kernel choice of the expert
// layer (forward, bwd_data, bwd_weight).
#include <algorithm>
#include <cstdint>
#include <new>
#include <string>

#include "cbd_internal.h"
#include "expert_common.h"
#include "expert_internal.h"

namespace {

using cbd::ExpertArgs;
using cbd::ExpertLaunch;
using cbd::host::Block;
using cbd::host::esize;
using cbd::host::fail;
using cbd::host::guarded;
using cbd::host::kMaxGrid;
using cbd::host::kMaxSlice;
using cbd::host::kThreads;
using cbd::host::on16;
using cbd::host::share;

// Launch of an operator.  narrow_strides: 256 rows of either input stay within
// 32-bit offsets; dma: and both start every row on a 16-byte boundary;
// whole_out: the output's rows are 16-byte multiples on 16-byte boundaries.
ExpertLaunch choose(const cbd_expert_plan_s& plan, int op, bool narrow_strides, bool dma, bool whole_out) {
  const cbd_expert_problem& p = plan.prob;
  ExpertLaunch l;
  l.dtype = p.dtype;
  l.out_dtype = op == CBD_EXPERT_BWD_WEIGHT ? p.dw_dtype : p.dtype;
  l.form = op == CBD_EXPERT_BWD_WEIGHT ? cbd::EXPERT_DW
           : (op == CBD_EXPERT_FORWARD) == (p.w_layout == CBD_EXPERT_EKC) ? cbd::EXPERT_AK
                                                                          : cbd::EXPERT_AM;
  l.threads = kThreads;
  // The contiguous side of the output and, for bwd_weight, its other side.
  const bool wide_k = op == CBD_EXPERT_FORWARD || (op == CBD_EXPERT_BWD_WEIGHT && p.w_layout == CBD_EXPERT_ECK);
  const int64_t m = wide_k ? p.k : p.c;
  const int64_t n = wide_k ? p.c : p.k;
  auto grid = [&](int bm, int bn) -> int64_t {
    const int64_t tm = (m + bm - 1) / bm;
    if (op == CBD_EXPERT_BWD_WEIGHT) return tm * ((n + bn - 1) / bn) * p.experts;
    const int64_t spans = p.experts + 1 < p.tokens ? p.experts + 1 : p.tokens;
    return tm * (p.tokens / bn + spans);
  };
  l.kernel = plan.opt.force_kernel;
  // Few rows an expert: 64 experts of 2048 x 1408, stream / mfma in us at 16
  // rows an expert 90 / 95 (AK) and 68 / 77 (AM), at 32 rows 125 / 95 and 83 /
  // 79.  Experts whose weights the caches hold together are faster on mfma from
  // fewer rows on (2048 x 1024, AK, the same weights again and again: 57 / 40).
  const int stream_bm = l.form == cbd::EXPERT_AK ? 32 : 128;
  const bool stream_ok = op != CBD_EXPERT_BWD_WEIGHT && narrow_strides && grid(stream_bm, 32) <= kMaxGrid;
  if (l.kernel == CBD_EXPERT_KERNEL_AUTO)
    l.kernel = p.dtype != CBD_BF16 ? CBD_EXPERT_KERNEL_GENERIC
               : stream_ok && p.tokens <= (l.form == cbd::EXPERT_AK ? 16 : 24) * p.experts
                   ? CBD_EXPERT_KERNEL_STREAM
                   : CBD_EXPERT_KERNEL_MFMA;
  if (l.kernel == CBD_EXPERT_KERNEL_STREAM && !stream_ok) l.kernel = CBD_EXPERT_KERNEL_MFMA;
  l.dma = 0;
  if (l.kernel == CBD_EXPERT_KERNEL_STREAM) {
    l.bm = stream_bm;
    l.bn = 32;
    l.grid = grid(l.bm, l.bn);
    return l;
  }
  if (l.kernel == CBD_EXPERT_KERNEL_MFMA) {
    // k runs along the rows of x (dy), and of W in the AK form.
    l.dma = dma && (op == CBD_EXPERT_BWD_WEIGHT || n % 8 == 0);
    // 256 x 256 tiles where they fill the card twice and, with rows an expert
    // that vary, their last row tiles are few (256 / 128 in us, 64 experts of
    // 2048 inputs: 2048 outputs, 128 rows an expert 173 / 143, 192 rows 171 /
    // 187, 256 rows 182 / 201; 1024 outputs 99 / 76, 103 / 105, 104 / 109).  A
    // last feature tile that is at most half used takes more rows to be worth
    // it (1408 outputs: 256 rows 152 / 149, 384 rows 165 / 192).
    const bool half = (m + 127) / 128 % 2 != 0;
    const bool many = op == CBD_EXPERT_BWD_WEIGHT || p.tokens >= (half ? 384 : 192) * p.experts;
    l.bm = l.bn = l.dma && whole_out && many && grid(256, 256) >= 512 ? 256 : 128;
  } else {
    // 64 x 64 where 128 x 128 would leave compute units idle (64 / 128 in us: at
    // 320 tiles of 128 114 / 153, at 192 29 / 49) or compute a tenth more for
    // nothing (59801 rows, 176 wide: 849 / 1033; 320 wide 443 / 465); otherwise
    // they are alike (256 wide 1090 / 1063, 2048 wide 716 / 748).
    auto covered = [&](int64_t b) {
      return (m + b - 1) / b * b * (op == CBD_EXPERT_BWD_WEIGHT ? (n + b - 1) / b * b : 1);
    };
    const bool small = grid(128, 128) < 512 || covered(128) * 10 > covered(64) * 11;
    l.bm = l.bn = small && grid(64, 64) <= kMaxGrid ? 64 : 128;
  }
  l.grid = grid(l.bm, l.bn);
  // Workgroups that stay: one (256 x 256: its LDS) or two a compute unit.
  if (l.kernel == CBD_EXPERT_KERNEL_MFMA && l.grid <= INT32_MAX)
    l.grid = std::min<int64_t>(l.grid, l.bm == 256 ? 256 : 512);
  return l;
}

cbd_status check_op(const cbd_expert_plan_t* plan, const void* row_in, const void* second, const void* ends,
                    const void* out, int op) {
  if (!plan || !ends) return fail(CBD_ERR_INVALID_ARG, "NULL plan or ends");
  const bool rows = plan->prob.tokens > 0;
  // Row tensors of a call with no rows may be NULL; weights may not.
  const bool row_missing = rows && (!row_in || (op == CBD_EXPERT_BWD_WEIGHT ? !second : !out));
  const bool w_missing = op == CBD_EXPERT_BWD_WEIGHT ? !out : !second;
  if (row_missing || w_missing) return fail(CBD_ERR_INVALID_ARG, "NULL tensor pointer");
  return CBD_OK;
}

// row_in: x / dy; second: W, or x for bwd_weight; out: y / dx / dW.
cbd_status run(const cbd_expert_plan_t* plan, int op, const void* row_in, const void* second, const void* ends,
               void* out, int32_t accumulate, const cbd_expert_strides* st, void* stream) {
  const cbd_status bad = check_op(plan, row_in, second, ends, out, op);
  if (bad != CBD_OK) return bad;
  const cbd_expert_problem& p = plan->prob;
  if (accumulate != 0 && accumulate != 1) return fail(CBD_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  cbd_expert_strides s = {0, 0, 0, 0};
  if (st) s = *st;
  const int64_t w_rows = p.w_layout == CBD_EXPERT_EKC ? p.k : p.c;
  const int64_t w_width = p.w_layout == CBD_EXPERT_EKC ? p.c : p.k;
  if (!s.x_row) s.x_row = p.c;
  if (!s.y_row) s.y_row = p.k;
  if (!s.w_row) s.w_row = w_width;
  if (!s.w_expert) s.w_expert = (w_rows - 1) * s.w_row + w_width;
  constexpr int64_t kMaxStride = int64_t(1) << 40;
  if (s.x_row < p.c || s.y_row < p.k || s.w_row < w_width)
    return fail(CBD_ERR_INVALID_ARG, "a row stride is smaller than the row");
  if (s.w_row > kMaxSlice || s.w_expert > kMaxStride || s.x_row > kMaxSlice || s.y_row > kMaxSlice)
    return fail(CBD_ERR_UNSUPPORTED, "a stride is too large");
  if (s.w_expert < (w_rows - 1) * s.w_row + w_width)
    return fail(CBD_ERR_INVALID_ARG, "the expert stride is smaller than an expert's slice");
  const int es = esize(p.dtype), wes = op == CBD_EXPERT_BWD_WEIGHT ? esize(p.dw_dtype) : es;
  // Tiles address with 32-bit offsets: 256 rows of a row tensor, one expert of W.
  if (s.x_row * 256 * es >= kMaxSlice || s.y_row * 256 * es >= kMaxSlice ||
      ((w_rows - 1) * s.w_row + w_width) * wes >= kMaxSlice)
    return fail(CBD_ERR_UNSUPPORTED, "a stride passes 32-bit offsets within a tile");

  const Block bx = {op == CBD_EXPERT_FORWARD ? row_in : op == CBD_EXPERT_BWD_DATA ? out : second,
                    p.tokens, p.c, s.x_row, 1, 0, es};
  const Block by = {op == CBD_EXPERT_FORWARD ? out : row_in, p.tokens, p.k, s.y_row, 1, 0, es};
  const Block bw = {op == CBD_EXPERT_BWD_WEIGHT ? out : second, w_rows, w_width, s.w_row, p.experts, s.w_expert,
                    wes};
  const Block be = {ends, 1, p.experts, p.experts, 1, 0, p.ends_bits / 8};
  if (((uintptr_t)bx.p | (uintptr_t)by.p) & (uintptr_t)(es - 1) || (uintptr_t)bw.p & (uintptr_t)(wes - 1) ||
      (uintptr_t)ends & (uintptr_t)(be.es - 1))
    return fail(CBD_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
  const Block& bo = op == CBD_EXPERT_FORWARD ? by : op == CBD_EXPERT_BWD_DATA ? bx : bw;
  for (const Block* b : {&bx, &by, &bw, &be})
    if (b != &bo && share(bo, *b)) return fail(CBD_ERR_INVALID_ARG, "the output overlaps an operand");

  if (p.tokens == 0 && (op != CBD_EXPERT_BWD_WEIGHT || accumulate)) {
    cbd::set_error("");
    return CBD_OK;
  }

  const bool whole_out = on16(bo) && bo.width % (16 / bo.es) == 0;
  bool dma = true, narrow_strides = true;
  for (const Block* b : {&bx, &by, &bw})
    if (b != &bo) {
      narrow_strides = narrow_strides && b->ld * 256 * b->es < kMaxSlice;
      dma = dma && on16(*b);
    }
  dma = dma && narrow_strides;
  const ExpertLaunch l = choose(*plan, op, narrow_strides, dma, whole_out);
  if (l.grid > kMaxGrid) return fail(CBD_ERR_UNSUPPORTED, "too many tiles for one launch");

  ExpertArgs a = {};
  a.ends = ends;
  a.ends64 = p.ends_bits == 64;
  a.T = (int32_t)p.tokens;
  a.E = (int32_t)p.experts;
  a.out = out;
  a.accumulate = accumulate;
  a.whole_out = whole_out;
  if (op == CBD_EXPERT_BWD_WEIGHT) {
    const Block& ba = p.w_layout == CBD_EXPERT_EKC ? bx : by;
    const Block& bb = p.w_layout == CBD_EXPERT_EKC ? by : bx;
    a.a = ba.p;
    a.lda = ba.ld;
    a.M = (int32_t)ba.width;
    a.b = bb.p;
    a.ldb = bb.ld;
    a.N = (int32_t)bb.width;
    a.ldo = s.w_row;
    a.o_expert = s.w_expert;
    a.tiles_n = (a.N + l.bn - 1) / l.bn;
  } else {
    const Block& bb = op == CBD_EXPERT_FORWARD ? bx : by;
    a.a = second;
    a.lda = s.w_row;
    a.a_expert = s.w_expert;
    a.M = (int32_t)bo.width;
    a.b = row_in;
    a.ldb = bb.ld;
    a.K = (int32_t)bb.width;
    a.ldo = bo.ld;
  }
  a.tiles_m = (a.M + l.bm - 1) / l.bm;
  const int err = l.kernel == CBD_EXPERT_KERNEL_MFMA     ? cbd::launch_expert_mfma(a, l, stream)
                  : l.kernel == CBD_EXPERT_KERNEL_STREAM ? cbd::launch_expert_stream(a, l, stream)
                                                         : cbd::launch_expert_generic(a, l, stream);
  if (err) {
    cbd::set_error(std::string("expert kernel launch failed: ") + cbd::hip_error_name(err));
    return CBD_ERR_HIP;
  }
  cbd::set_error("");
  return CBD_OK;
}

cbd_status make_plan(const cbd_expert_problem* q, const cbd_expert_options* opt, cbd_expert_plan_t** out) {
  if (!q || !out) return fail(CBD_ERR_INVALID_ARG, "NULL problem or output");
  *out = nullptr;
  if (q->tokens < 0 || q->experts < 1 || q->c < 1 || q->k < 1)
    return fail(CBD_ERR_INVALID_ARG, "tokens must be >= 0, experts, c and k >= 1");
  if (q->w_layout != CBD_EXPERT_EKC && q->w_layout != CBD_EXPERT_ECK)
    return fail(CBD_ERR_INVALID_ARG, "unknown w_layout");
  if (q->dtype != CBD_F32 && q->dtype != CBD_BF16) return fail(CBD_ERR_INVALID_ARG, "unknown dtype");
  if (q->dw_dtype != CBD_F32 && !(q->dw_dtype == CBD_BF16 && q->dtype == CBD_BF16))
    return fail(CBD_ERR_INVALID_ARG, "dw_dtype must be f32, or bf16 with bf16 operands");
  if (q->ends_bits != 32 && q->ends_bits != 64) return fail(CBD_ERR_INVALID_ARG, "ends_bits must be 32 or 64");
  if (opt) {
    if (opt->force_kernel < CBD_EXPERT_KERNEL_AUTO || opt->force_kernel > CBD_EXPERT_KERNEL_STREAM)
      return fail(CBD_ERR_INVALID_ARG, "unknown force_kernel");
    for (int32_t r : opt->reserved)
      if (r) return fail(CBD_ERR_INVALID_ARG, "reserved options must be zero");
    if (opt->force_kernel > CBD_EXPERT_KERNEL_GENERIC && q->dtype != CBD_BF16)
      return fail(CBD_ERR_UNSUPPORTED, "the forced kernel takes bf16 operands only");
  }
  if (q->experts > 65536) return fail(CBD_ERR_UNSUPPORTED, "more than 65536 experts");
  if (q->tokens > (int64_t(1) << 30)) return fail(CBD_ERR_UNSUPPORTED, "more than 2^30 tokens");
  if (q->c > (1 << 20) || q->k > (1 << 20)) return fail(CBD_ERR_UNSUPPORTED, "c or k above 2^20");
  const int64_t slice = q->c * q->k;
  if (slice * esize(q->dtype) >= kMaxSlice || slice * esize(q->dw_dtype) >= kMaxSlice)
    return fail(CBD_ERR_UNSUPPORTED, "an expert's weights take 2^31 bytes or more");
  cbd_expert_plan_s* p = new (std::nothrow) cbd_expert_plan_s;
  if (!p) return fail(CBD_ERR_NO_MEMORY, "out of host memory");
  p->prob = *q;
  p->opt = opt ? *opt : cbd_expert_options{CBD_EXPERT_KERNEL_AUTO, {0, 0, 0}};
  *out = p;
  cbd::set_error("");
  return CBD_OK;
}

}  // namespace

extern "C" cbd_status cbd_expert_plan(const cbd_expert_problem* problem, const cbd_expert_options* options,
                                      cbd_expert_plan_t** out_plan) {
  return guarded([&] { return make_plan(problem, options, out_plan); });
}

extern "C" void cbd_expert_plan_destroy(cbd_expert_plan_t* plan) { delete plan; }

extern "C" cbd_status cbd_expert_plan_info(const cbd_expert_plan_t* plan, int32_t op, cbd_expert_info_t* out) {
  return guarded([&]() -> cbd_status {
    if (!plan || !out) return fail(CBD_ERR_INVALID_ARG, "NULL plan or output");
    if (op < CBD_EXPERT_FORWARD || op > CBD_EXPERT_BWD_WEIGHT) return fail(CBD_ERR_INVALID_ARG, "unknown op");
    const cbd_expert_problem& p = plan->prob;
    // Dense rows are 16-byte multiples when the widths are.
    const int64_t q = 16 / esize(p.dtype);
    const bool whole = p.c % q == 0 && p.k % q == 0;
    const ExpertLaunch l = choose(*plan, op, true, whole, whole);
    out->kernel = l.kernel;
    out->tile_m = l.bm;
    out->tile_n = l.bn;
    out->threads = l.threads;
    out->grid = l.grid;
    out->flops = 2 * p.tokens * p.c * p.k;
    cbd::set_error("");
    return CBD_OK;
  });
}

extern "C" cbd_status cbd_expert_forward(const cbd_expert_plan_t* plan, const void* x, const void* w,
                                         const void* ends, void* y, const cbd_expert_strides* strides,
                                         void* stream) {
  return guarded([&] { return run(plan, CBD_EXPERT_FORWARD, x, w, ends, y, 0, strides, stream); });
}

extern "C" cbd_status cbd_expert_bwd_data(const cbd_expert_plan_t* plan, const void* dy, const void* w,
                                          const void* ends, void* dx, const cbd_expert_strides* strides,
                                          void* stream) {
  return guarded([&] { return run(plan, CBD_EXPERT_BWD_DATA, dy, w, ends, dx, 0, strides, stream); });
}

extern "C" cbd_status cbd_expert_bwd_weight(const cbd_expert_plan_t* plan, const void* dy, const void* x,
                                            const void* ends, void* dw, int32_t accumulate,
                                            const cbd_expert_strides* strides, void* stream) {
  return guarded([&] { return run(plan, CBD_EXPERT_BWD_WEIGHT, dy, x, ends, dw, accumulate, strides, stream); });
}
