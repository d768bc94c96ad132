// gate_device.h -- the activation of a gated block, and which gate and other
// projection meet in a tile.
//
// All three activations are g times a step s(g) that rises from 0 to 1:
//   silu  s = 1 / (1 + exp(-g))
//   gelu  s = 1 / (1 + exp(-2 sqrt(2 / pi) (g + 0.044715 g^3)))   ((1 + tanh v) / 2)
//   relu  s = 1 where g > 0, else 0
// so with t = g (alpha + beta g^2) the derivative is s + s (1 - s) g t'(g).
#pragma once
#include "cbd_device.h"
#include "gated_internal.h"

namespace cbd {
namespace dev {

struct Gate {
  float alpha, beta;
  bool relu;

  __device__ inline explicit Gate(int act) {
    relu = act == CBD_ACT_RELU;
    alpha = act == CBD_ACT_GELU ? 1.5957691216057308f : 1.f;  // 2 sqrt(2 / pi)
    beta = act == CBD_ACT_GELU ? 1.5957691216057308f * 0.044715f : 0.f;
  }
  // g^2, kept finite: beta is 0 for silu.
  __device__ static inline float square(float g) { return __builtin_fminf(g * g, 3e38f); }
  // FINE: for f32 results; otherwise by the hardware's exp2 and reciprocal
  // (some 2^-21, against bf16's 2^-9).
  template <bool FINE>
  __device__ inline float step(float g) const {
    const float t = g * __builtin_fmaf(beta, square(g), alpha);
    const float s = FINE ? 1.f / (1.f + expf(-t))
                         : __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * t));
    return relu ? (g > 0.f ? 1.f : 0.f) : s;
  }
  // By comparison, so that relu of minus infinity is 0 and of NaN NaN.
  __device__ inline float times(float g, float s) const { return relu ? (g <= 0.f ? 0.f : g) : g * s; }
  template <bool FINE>
  __device__ inline float act(float g) const {
    return times(g, step<FINE>(g));
  }
  // The activation and its derivative.  Far out s (1 - s) is 0 and t'(g) may be
  // infinite: their product counts as 0.
  template <bool FINE>
  __device__ inline float act(float g, float& slope) const {
    const float s = step<FINE>(g);
    const float bend = s * (1.f - s);
    slope = bend == 0.f ? s : __builtin_fmaf(bend * g, __builtin_fmaf(3.f * beta, square(g), alpha), s);
    return times(g, s);
  }
};

// For bf16 results, one activation at a time: half the instructions of the
// general form, by the hardware's exp2 and reciprocal.  f(kind) is called with
// one of these.
template <int ACT>
struct GateOf {
  static constexpr float A = ACT == CBD_ACT_GELU ? 1.5957691216057308f : 1.f, B = A * 0.044715f, LOG2E = 1.4426950408889634f;
  __device__ static inline float act(float g, float* slope = nullptr) {
    if constexpr (ACT == CBD_ACT_RELU) {
      if (slope) *slope = g > 0.f ? 1.f : 0.f;
      return g <= 0.f ? 0.f : g;
    } else {
      float t = -LOG2E * g, bend = 1.f;  // -t log2(e), and t'(g)
      if constexpr (ACT == CBD_ACT_GELU) {
        const float q = Gate::square(g);
        t = g * __builtin_fmaf(-B * LOG2E, q, -A * LOG2E);
        bend = __builtin_fmaf(3.f * B, q, A);
      }
      const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t)), v = g * s;
      if (slope) *slope = __builtin_fmaf(v * (1.f - s), bend, s);
      return v;
    }
  }
};
template <typename F>
CBD_INLINE __device__ inline void with_gate(int act, F&& f) {
  if (act == CBD_ACT_SILU)
    f(GateOf<CBD_ACT_SILU>());
  else if (act == CBD_ACT_GELU)
    f(GateOf<CBD_ACT_GELU>());
  else
    f(GateOf<CBD_ACT_RELU>());
}

// Row r of an operand tile of F rows that holds two projections, for W waves
// side by side: every wave has F / W rows, first those of the gate, then the
// same features of the other projection.
template <int F, int W>
struct Pair {
  static constexpr int HALF = F / W / 2;
  __device__ static constexpr int feat(int r) { return r / (2 * HALF) * HALF + r % HALF; }
  __device__ static constexpr int part(int r) { return r / HALF & 1; }
};

}  // namespace dev
}  // namespace cbd
