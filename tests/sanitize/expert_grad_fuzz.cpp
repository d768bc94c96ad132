// Host fuzz of the expert layer's and the gradient operators' entry points for
// a sanitizer build: random problems, options, strides and addresses.  The
// launchers are replaced by checks of what they are handed; every call returns
// a status, nothing is launched on an error, and what is launched keeps to the
// limits that the kernels rely on.  Built with -fsanitize=address,undefined by
// tests/test_host_sanitizers.py together with the two sources.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <string>
#include <vector>

#include "cbd_internal.h"
#include "expert_internal.h"
#include "grad_internal.h"

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

static int expert(const ExpertArgs& a, const ExpertLaunch& l, int kernel) {
  launches++;
  expect(l.kernel == kernel && l.grid >= 1 && l.grid < (int64_t(1) << 24), "grid");
  expect(a.E >= 1 && a.T >= 0 && a.M >= 1 && a.tiles_m == (a.M + l.bm - 1) / l.bm, "sizes");
  expect(l.form == EXPERT_DW ? a.N >= 1 : a.K >= 1 && a.T >= 1, "contracted side");
  expect(a.lda >= 1 && a.ldb >= 1 && a.ldo >= a.M, "strides");
  const int64_t es = l.dtype == CBD_F32 ? 4 : 2, os = l.out_dtype == CBD_F32 ? 4 : 2;
  expect(a.ldb * 256 * es < (int64_t(1) << 31), "rows of a tile pass 32-bit offsets");
  expect((l.form == EXPERT_DW ? (int64_t)(a.N - 1) * a.ldo + a.M : a.ldo * 256) * os < (int64_t(1) << 31),
         "results of a tile pass 32-bit offsets");
  expect(((uintptr_t)a.out & (os - 1)) == 0 && ((uintptr_t)a.ends & (a.ends64 ? 7 : 3)) == 0, "alignment");
  if (l.dma) {
    expect((((uintptr_t)a.a | (uintptr_t)a.b) & 15) == 0 && a.lda % 8 == 0 && a.ldb % 8 == 0, "16-byte rows");
    expect(a.lda * 256 * es < (int64_t(1) << 31), "rows of an operand pass 32-bit offsets");
    expect(l.form == EXPERT_DW || a.K % 8 == 0, "16-byte steps");
  }
  if (a.whole_out) expect(((uintptr_t)a.out & 15) == 0 && a.ldo * os % 16 == 0 && a.M * os % 16 == 0, "whole results");
  if (l.kernel == CBD_EXPERT_KERNEL_MFMA) {
    expect(l.dtype == CBD_BF16 && l.bm == l.bn && (l.bm == 128 || (l.bm == 256 && l.dma && a.whole_out)), "tile");
    const int64_t tiles = l.form == EXPERT_DW ? (int64_t)a.tiles_m * a.tiles_n * a.E
                                              : (int64_t)a.tiles_m * (a.T / l.bn + std::min(a.E + 1, a.T));
    expect(tiles <= INT32_MAX && (l.grid == tiles || l.grid == (l.bm == 256 ? 256 : 512)), "workgroups that stay");
  }
  if (l.kernel == CBD_EXPERT_KERNEL_STREAM)
    expect(l.dtype == CBD_BF16 && l.form != EXPERT_DW && a.lda * 256 * es < (int64_t(1) << 31), "stream");
  return 0;
}
int launch_expert_generic(const ExpertArgs& a, const ExpertLaunch& l, void*) {
  return expert(a, l, CBD_EXPERT_KERNEL_GENERIC);
}
int launch_expert_mfma(const ExpertArgs& a, const ExpertLaunch& l, void*) { return expert(a, l, CBD_EXPERT_KERNEL_MFMA); }
int launch_expert_stream(const ExpertArgs& a, const ExpertLaunch& l, void*) {
  return expert(a, l, CBD_EXPERT_KERNEL_STREAM);
}

static uint64_t workspace;
static int64_t bytes_passed;
static int batch(const GradArgs& a) {
  launches++;
  expect(a.n >= 1 && a.n <= kGradBatch, "tensors of a launch");
  uint64_t chunks = 0;
  for (int i = 0; i < a.n; i++) {
    const uint64_t bytes = (uint64_t)a.t[i].count * (a.t[i].dtype == CBD_F32 ? 4 : 2);
    expect(a.t[i].in && a.t[i].out && a.t[i].count > 0 && a.t[i].chunk_begin == chunks, "entry");
    chunks += (bytes + kGradChunkBytes - 1) / kGradChunkBytes;
    bytes_passed += (int64_t)bytes;
  }
  expect(chunks == a.chunks, "chunks");
  return 0;
}
int launch_grad_partial(const GradArgs& a, uint32_t grid, void*) {
  expect(grid >= 1 && grid <= (uint32_t)kGradMaxGrid && a.first + grid <= a.partials, "partial sums");
  expect((uint64_t)a.partials * 8 <= workspace, "workspace");
  return batch(a);
}
int launch_grad_scale(const GradArgs& a, uint32_t grid, void*) {
  expect(grid >= 1 && grid <= (uint32_t)kGradMaxGrid, "grid");
  return batch(a);
}
int launch_grad_small(const GradArgs& a, int, void*) { return batch(a); }
int launch_grad_finish(const GradArgs& a, void*) {
  launches++;
  expect(a.norm && (uint64_t)a.partials * 8 <= workspace, "finish");
  return 0;
}
}  // namespace cbd

template <typename R>
static int64_t pick(R& rng, std::initializer_list<int64_t> v) {
  return *(v.begin() + rng() % v.size());
}

static void experts(std::mt19937_64& rng, long iters) {
  auto uni = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  for (long it = 0; it < iters; it++) {
    cbd_expert_problem p = {};
    p.tokens = rng() % 8 ? uni(0, 70000) : pick(rng, {-1, 0, 1, 1 << 20, 1 << 30, (int64_t)1 << 31});
    p.experts = rng() % 8 ? uni(1, 130) : pick(rng, {0, 1, 65536, 65537});
    p.c = rng() % 8 ? uni(1, 5000) : pick(rng, {0, 1, 8, 1 << 20, (1 << 20) + 1});
    p.k = rng() % 8 ? uni(1, 5000) : pick(rng, {0, 1, 8, 1 << 20, (1 << 20) + 1});
    if (rng() % 2) p.c = (p.c + 7) / 8 * 8, p.k = (p.k + 7) / 8 * 8;
    p.w_layout = (int32_t)(rng() % 40 ? uni(0, 1) : 2);
    p.dtype = (int32_t)(rng() % 40 ? uni(0, 1) : 5);
    p.dw_dtype = (int32_t)(rng() % 40 ? uni(0, 1) : -1);
    p.ends_bits = (int32_t)(rng() % 40 ? pick(rng, {32, 64}) : 16);
    cbd_expert_options o = {(int32_t)uni(-1, 2), {0, 0, 0}};
    if (rng() % 50 == 0) o.reserved[rng() % 3] = 1;
    cbd_expert_plan_t* plan = nullptr;
    const cbd_status st = cbd_expert_plan(&p, rng() % 3 ? nullptr : &o, &plan);
    expect((st == CBD_OK) == (plan != nullptr), "a status and its plan");
    if (!plan) continue;
    for (int op = 0; op < 3; op++) {
      cbd_expert_info_t info;
      expect(cbd_expert_plan_info(plan, op, &info) == CBD_OK, "info");
    }
    // Three regions far apart, sometimes moved onto one another.
    uint64_t at[4];
    for (int i = 0; i < 4; i++) at[i] = ((uint64_t)(i + 1) << 56) + 16 * (rng() % 64);
    if (rng() % 4 == 0) at[rng() % 4] += pick(rng, {1, 2, 4, 8});
    if (rng() % 10 == 0) at[rng() % 4] = at[rng() % 4] + 2 * (rng() % 9000);
    if (rng() % 40 == 0) at[rng() % 4] = 0;
    const int64_t wr = p.w_layout == CBD_EXPERT_EKC ? p.k : p.c, ww = p.w_layout == CBD_EXPERT_EKC ? p.c : p.k;
    cbd_expert_strides s = {};
    if (rng() % 2) s.x_row = p.c + pick(rng, {-1, 0, 1, 8, 64, 1 << 22, (int64_t)1 << 40});
    if (rng() % 2) s.y_row = p.k + pick(rng, {0, 1, 8, 64, 1 << 22});
    if (rng() % 2) s.w_row = ww + pick(rng, {-1, 0, 1, 8, 64, 1 << 20});
    if (rng() % 2) s.w_expert = (wr - 1) * (s.w_row ? s.w_row : ww) + ww + pick(rng, {-1, 0, 1, 8, 64, (int64_t)1 << 41});
    const cbd_expert_strides* sp = rng() % 2 ? &s : nullptr;
    auto ptr = [&](int i) { return (void*)(uintptr_t)at[i]; };
    for (int op = 0; op < 3; op++) {
      const long before = launches;
      const cbd_status r =
          op == 0   ? cbd_expert_forward(plan, ptr(0), ptr(1), ptr(2), ptr(3), sp, nullptr)
          : op == 1 ? cbd_expert_bwd_data(plan, ptr(0), ptr(1), ptr(2), ptr(3), sp, nullptr)
                    : cbd_expert_bwd_weight(plan, ptr(0), ptr(1), ptr(2), ptr(3), (int32_t)pick(rng, {0, 0, 1, 1, 2}), sp,
                                            nullptr);
      expect(r == CBD_OK ? launches <= before + 1 : launches == before, "a launch after an error");
      expect(r == CBD_OK || r == CBD_ERR_INVALID_ARG || r == CBD_ERR_UNSUPPORTED, "status");
    }
    cbd_expert_plan_destroy(plan);
  }
}

static void grads(std::mt19937_64& rng, long iters) {
  auto uni = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  for (long it = 0; it < iters; it++) {
    const int n = (int)(rng() % 20 ? uni(0, 12) : uni(100, 400));
    std::vector<int64_t> counts(n);
    std::vector<int32_t> types(n);
    for (int i = 0; i < n; i++) {
      counts[i] = rng() % 10 ? uni(0, 3000000) : pick(rng, {0, 1, (int64_t)1 << 33});
      types[i] = (int32_t)uni(0, 1);
    }
    if (n && rng() % 40 == 0) counts[rng() % n] = pick(rng, {-1, (int64_t)1 << 40});
    if (n && rng() % 40 == 0) types[rng() % n] = 3;
    cbd_grad_plan_t* plan = nullptr;
    const cbd_status st = cbd_grad_plan(counts.data(), types.data(), n, &plan);
    expect((st == CBD_OK) == (plan != nullptr), "a status and its plan");
    if (!plan) continue;
    expect(cbd_grad_workspace_size(plan, &cbd::workspace) == CBD_OK && cbd::workspace % 256 == 0, "workspace size");
    std::vector<void*> in(n), out(n);
    std::vector<uint64_t> size(n);
    uint64_t a = 1 << 20, b = (uint64_t)1 << 60;
    for (int i = 0; i < n; i++) {
      size[i] = (uint64_t)counts[i] * (types[i] == CBD_F32 ? 4 : 2);
      a += 4 * (rng() % 3);
      b += 4 * (rng() % 3);
      in[i] = (void*)a;
      out[i] = rng() % 3 ? (void*)b : (void*)a;
      a += (size[i] + 3) / 4 * 4;
      b += (size[i] + 3) / 4 * 4;
    }
    if (n && rng() % 4 == 0) (rng() % 2 ? in : out)[rng() % n] = (char*)(rng() % 2 ? in : out)[rng() % n] + uni(-2, 2) * 2;
    if (n && rng() % 40 == 0) in[rng() % n] = nullptr;
    const bool clip = rng() % 3 != 0, place = rng() % 2 == 0;
    uint64_t norm = (uint64_t)1 << 61, ws = (uint64_t)3 << 60;
    if (n && rng() % 20 == 0) norm = (uint64_t)in[rng() % n];
    // Whether something that is written overlaps something else, pair by pair.
    struct R {
      uint64_t p, n;
      bool w;
      int own;
    };
    std::vector<R> r = {{norm, 4, true, -1}, {ws, cbd::workspace, true, -2}};
    bool null = false, odd = (norm & 3) != 0;
    for (int i = 0; i < n; i++) {
      if (!size[i]) continue;
      const uint64_t mask = types[i] == CBD_F32 ? 3 : 1, x = (uint64_t)in[i];
      const uint64_t y = clip ? (uint64_t)(place ? in[i] : out[i]) : 0;
      null = null || !x || (clip && !y);
      odd = odd || (x & mask) || (y & mask);
      if (x != y) r.push_back({x, size[i], false, i});
      if (clip) r.push_back({y, size[i], true, i});
    }
    bool overlap = false;
    if (r.size() < 60)
      for (size_t i = 0; i < r.size(); i++)
        for (size_t j = 0; j < i; j++)
          overlap = overlap || ((r[i].w || r[j].w) && r[i].p < r[j].p + r[j].n && r[j].p < r[i].p + r[i].n);
    const long before = launches;
    cbd::bytes_passed = 0;
    const cbd_status s =
        clip ? cbd_grad_clip(plan, in.data(), place ? nullptr : out.data(), 1.0, (float*)norm, (void*)ws, cbd::workspace, nullptr)
             : cbd_grad_norm(plan, in.data(), (float*)norm, (void*)ws, cbd::workspace, nullptr);
    if (r.size() < 60) expect((s == CBD_OK) == (!null && !odd && !overlap), "overlaps and alignment");
    expect(s == CBD_OK || launches == before, "a launch after an error");
    if (s == CBD_OK) {
      int64_t total = 0;
      for (uint64_t v : size) total += (int64_t)v;
      const int64_t times = launches - before == 1 || !clip ? 1 : 2;
      expect(cbd::bytes_passed == total * (total ? times : 1), "every tensor in every pass");
    }
    cbd_grad_plan_destroy(plan);
  }
}

int main(int argc, char** argv) {
  const long iters = argc > 1 ? std::atol(argv[1]) : 10000;
  std::mt19937_64 rng(argc > 2 ? std::atoll(argv[2]) : 1);
  experts(rng, iters);
  const long expert_launches = launches;
  grads(rng, iters / 4);
  std::printf("launches: %ld experts, %ld gradients; checks: %ld\n", expert_launches, launches - expert_launches, checked);
  return broken || expert_launches < iters / 10 || launches - expert_launches < iters / 10;
}
