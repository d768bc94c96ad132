// gated_api.cpp -- argument checks and kernel choice of the gated experts.
#include <algorithm>
#include <cstdint>
#include <string>

#include "cbd_internal.h"
#include "expert_common.h"
#include "gated_internal.h"

namespace {

using cbd::ExpertLaunch;
using cbd::GatedArgs;
using cbd::host::Block;
using cbd::host::esize;
using cbd::host::fail;
using cbd::host::guarded;
using cbd::host::kMaxGrid;
using cbd::host::kMaxSlice;
using cbd::host::on16;
using cbd::host::share;

// Width of h: half of the projections' outputs, or the last one's inputs.
int64_t hidden(const cbd_expert_problem& p, bool bwd) { return bwd ? p.c : p.k / 2; }

// narrow_strides: 256 rows of any input stay within 32-bit offsets; dma: the
// operands' rows (and the second projection's features) start on 16-byte
// boundaries; whole_out: so do all rows of the other tensors, in 16-byte
// multiples.  bm counts features of h.
ExpertLaunch choose(const cbd_expert_plan_s& plan, bool bwd, bool narrow_strides, bool dma, bool whole_out) {
  const cbd_expert_problem& p = plan.prob;
  ExpertLaunch l;
  l.dtype = l.out_dtype = p.dtype;
  l.form = bwd == (p.w_layout == CBD_EXPERT_ECK) ? cbd::EXPERT_AK : cbd::EXPERT_AM;
  l.threads = cbd::host::kThreads;
  const int64_t m = hidden(p, bwd), n = bwd ? p.k : p.c;
  const int parts = bwd ? 1 : 2;  // projections in a tile of weights
  auto grid = [&](int64_t bm, int64_t bn) -> int64_t {
    const int64_t spans = p.experts + 1 < p.tokens ? p.experts + 1 : p.tokens;
    return (m + bm - 1) / bm * (p.tokens / bn + spans);
  };
  l.kernel = plan.opt.force_kernel;
  // Few rows an expert: 64 experts of 2048 inputs and 2 x 1408 outputs, stream /
  // mfma in us at 8, 16, 20 and 32 rows an expert 142 / 168, 169 / 171, 186 / 172
  // and 235 / 175 (AK), 128 / 131, 133 / 134, 140 / 136 and 158 / 141 (AM; alike up
  // to 24, as for the expert products).
  const int stream_bm = (l.form == cbd::EXPERT_AK ? 32 : 128) / 2;
  const bool stream_ok = !bwd && narrow_strides && grid(stream_bm, 32) <= kMaxGrid;
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
  int64_t tile;
  if (l.kernel == CBD_EXPERT_KERNEL_MFMA) {
    l.dma = dma && n % 8 == 0;
    // 256 x 256 tiles by the rule of the expert products, whose features these
    // `parts * m` are (256 / 128 in us, forward: 64 experts of 2048 inputs and 2 x
    // 1408 outputs at 160 rows an expert 232 / 213, 192 228 / 234, 256 259 / 292,
    // 384 340 / 389, 32 of 2048 and 2 x 1024 at 256 rows 104 / 107; backward, 1408
    // features, whose last tile of 256 is half used, at 256 rows 205 / 184, 384
    // 242 / 238).
    const bool half = (parts * m + 127) / 128 % 2 != 0;
    const bool many = p.tokens >= (half ? 384 : 192) * p.experts;
    tile = l.dma && whole_out && many && grid(256 / parts, 256) >= 512 ? 256 : 128;
  } else {
    // 64 x 64 (of the expert products' two tiles: 64 / 128 in us, f32, 4 experts,
    // 16384 rows, 2048 inputs, 2 x 2048 outputs 2354 / 2308 and backward 1306 /
    // 1309; 8192 rows, 2 x 1024 572 / 627 and 342 / 423; 8 experts, 4096 rows, 1024
    // inputs, 2 x 1024 165 / 197 and 105 / 151; 64 experts, 8192 rows, 2 x 704 247 /
    // 332 and 154 / 219).
    tile = 64;
  }
  l.bm = (int32_t)(tile / parts);
  l.bn = (int32_t)tile;
  l.grid = grid(l.bm, l.bn);
  // Workgroups that stay: one (256 x 256: its LDS) or two a compute unit.
  if (l.kernel == CBD_EXPERT_KERNEL_MFMA && l.grid <= INT32_MAX)
    l.grid = std::min<int64_t>(l.grid, tile == 256 ? 256 : 512);
  return l;
}

// rows: x or dy; out: h or dgu; gu: written (forward, may be NULL) or read.
cbd_status run(const cbd_expert_plan_t* plan, bool bwd, const void* rows, const void* w, const void* gu_in,
               const void* ends, void* out, void* gu_out, int32_t act, const cbd_gated_strides* st, void* stream) {
  if (!plan || !ends || !w) return fail(CBD_ERR_INVALID_ARG, "NULL plan, ends or weights");
  const cbd_expert_problem& p = plan->prob;
  if (act < CBD_ACT_SILU || act > CBD_ACT_RELU) return fail(CBD_ERR_INVALID_ARG, "unknown activation");
  if (!bwd && p.k % 2) return fail(CBD_ERR_INVALID_ARG, "two projections need a plan with even k");
  const void* const gu = bwd ? gu_in : gu_out;
  if (p.tokens > 0 && (!rows || !out || (bwd && !gu))) return fail(CBD_ERR_INVALID_ARG, "NULL tensor pointer");
  const int64_t m = hidden(p, bwd), wide_in = bwd ? p.k : p.c;
  const int64_t w_rows = p.w_layout == CBD_EXPERT_EKC ? p.k : p.c;
  const int64_t w_width = p.w_layout == CBD_EXPERT_EKC ? p.c : p.k;
  cbd_gated_strides s = {0, 0, 0, 0, 0, 0};
  if (st) s = *st;
  if (!s.in_row) s.in_row = wide_in;
  if (!s.h_row) s.h_row = m;
  if (!s.gu_row) s.gu_row = 2 * m;
  if (!s.dgu_row) s.dgu_row = 2 * m;
  if (!s.w_row) s.w_row = w_width;
  if (!s.w_expert) s.w_expert = (w_rows - 1) * s.w_row + w_width;
  if (s.in_row < wide_in || s.h_row < m || s.gu_row < 2 * m || s.dgu_row < 2 * m || s.w_row < w_width)
    return fail(CBD_ERR_INVALID_ARG, "a row stride is smaller than the row");
  constexpr int64_t kMaxStride = int64_t(1) << 40;
  for (int64_t v : {s.in_row, s.h_row, s.gu_row, s.dgu_row, s.w_row})
    if (v > kMaxSlice) return fail(CBD_ERR_UNSUPPORTED, "a stride is too large");
  if (s.w_expert > kMaxStride) return fail(CBD_ERR_UNSUPPORTED, "a stride is too large");
  if (s.w_expert < (w_rows - 1) * s.w_row + w_width)
    return fail(CBD_ERR_INVALID_ARG, "the expert stride is smaller than an expert's slice");
  const int es = esize(p.dtype);
  const int64_t out_row = bwd ? s.dgu_row : s.h_row, out_width = bwd ? 2 * m : m;
  // Tiles address with 32-bit offsets: 256 rows of a row tensor, one expert of W.
  for (int64_t v : {s.in_row, out_row, gu ? s.gu_row : 0})
    if (v * 256 * es >= kMaxSlice) return fail(CBD_ERR_UNSUPPORTED, "a stride passes 32-bit offsets within a tile");
  if (((w_rows - 1) * s.w_row + w_width) * es >= kMaxSlice)
    return fail(CBD_ERR_UNSUPPORTED, "a stride passes 32-bit offsets within a tile");

  const Block bi = {rows, p.tokens, wide_in, s.in_row, 1, 0, es};
  const Block bo = {out, p.tokens, out_width, out_row, 1, 0, es};
  const Block bg = {gu, gu ? p.tokens : 0, 2 * m, s.gu_row, 1, 0, es};
  const Block bw = {w, w_rows, w_width, s.w_row, p.experts, s.w_expert, es};
  const Block be = {ends, 1, p.experts, p.experts, 1, 0, p.ends_bits / 8};
  for (const Block* b : {&bi, &bo, &bg, &bw, &be})
    if ((uintptr_t)b->p & (uintptr_t)(b->es - 1))
      return fail(CBD_ERR_UNSUPPORTED, "a pointer is not aligned to its element size");
  for (const Block* b : {&bi, &bg, &bw, &be})
    if (share(bo, *b)) return fail(CBD_ERR_INVALID_ARG, "the output overlaps another tensor");
  if (!bwd && gu)
    for (const Block* b : {&bi, &bw, &be})
      if (share(bg, *b)) return fail(CBD_ERR_INVALID_ARG, "gu overlaps another tensor");
  if (p.tokens == 0) {
    cbd::set_error("");
    return CBD_OK;
  }

  const int64_t up = p.w_layout == CBD_EXPERT_EKC ? m * s.w_row : m;  // forward only
  const bool narrow_strides = bi.ld * 256 * es < kMaxSlice && bw.ld * 256 * es < kMaxSlice;
  const bool dma = narrow_strides && on16(bi) && on16(bw) && (bwd || up * es % 16 == 0);
  const bool whole_out = on16(bo) && m * es % 16 == 0 && (!gu || on16(bg));
  const ExpertLaunch l = choose(*plan, bwd, narrow_strides, dma, whole_out);
  if (l.grid > kMaxGrid) return fail(CBD_ERR_UNSUPPORTED, "too many tiles for one launch");

  GatedArgs a = {};
  a.ends = ends;
  a.ends64 = p.ends_bits == 64;
  a.T = (int32_t)p.tokens;
  a.E = (int32_t)p.experts;
  a.out = out;
  a.whole_out = whole_out;
  a.a = w;
  a.lda = s.w_row;
  a.a_expert = s.w_expert;
  a.M = (int32_t)m;
  a.b = rows;
  a.ldb = s.in_row;
  a.K = (int32_t)wide_in;
  a.ldo = out_row;
  a.tiles_m = (a.M + l.bm - 1) / l.bm;
  a.gu = const_cast<void*>(gu);
  a.ldgu = s.gu_row;
  a.up = up;
  a.act = act;
  const int mode = bwd ? cbd::GATE_BWD : gu ? cbd::GATE_FWD_SAVE : cbd::GATE_FWD;
  const int err = l.kernel == CBD_EXPERT_KERNEL_MFMA     ? cbd::launch_gated_mfma(a, l, mode, stream)
                  : l.kernel == CBD_EXPERT_KERNEL_STREAM ? cbd::launch_gated_stream(a, l, mode, stream)
                                                         : cbd::launch_gated_generic(a, l, mode, stream);
  if (err) {
    cbd::set_error(std::string("gated expert kernel launch failed: ") + cbd::hip_error_name(err));
    return CBD_ERR_HIP;
  }
  cbd::set_error("");
  return CBD_OK;
}

}  // namespace

extern "C" cbd_status cbd_expert_gated_forward(const cbd_expert_plan_t* plan, const void* x, const void* w,
                                               const void* ends, void* h, void* gu, int32_t act,
                                               const cbd_gated_strides* strides, void* stream) {
  return guarded([&] { return run(plan, false, x, w, nullptr, ends, h, gu, act, strides, stream); });
}

extern "C" cbd_status cbd_expert_gated_bwd(const cbd_expert_plan_t* plan, const void* dy, const void* w,
                                           const void* gu, const void* ends, void* dgu, int32_t act,
                                           const cbd_gated_strides* strides, void* stream) {
  return guarded([&] { return run(plan, true, dy, w, gu, ends, dgu, nullptr, act, strides, stream); });
}

extern "C" cbd_status cbd_expert_gated_info(const cbd_expert_plan_t* plan, int32_t bwd, cbd_expert_info_t* out) {
  return guarded([&]() -> cbd_status {
    if (!plan || !out) return fail(CBD_ERR_INVALID_ARG, "NULL plan or output");
    if (bwd != 0 && bwd != 1) return fail(CBD_ERR_INVALID_ARG, "bwd must be 0 or 1");
    const cbd_expert_problem& p = plan->prob;
    if (!bwd && p.k % 2) return fail(CBD_ERR_INVALID_ARG, "two projections need a plan with even k");
    const int64_t q = 16 / esize(p.dtype), m = hidden(p, bwd);
    const bool whole = p.c % q == 0 && p.k % q == 0 && m % q == 0;
    const ExpertLaunch l = choose(*plan, bwd, true, whole, whole);
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
