// gated_internal.h -- kernel arguments and launchers of the gated experts.
#pragma once
#include "expert_internal.h"

namespace cbd {

// What the epilogue of a product does.
//   GATE_FWD       out = act(gate) * other; W holds both projections
//   GATE_FWD_SAVE  and both projections to gu
//   GATE_BWD       the product is dh: out = (dh * u * act'(g), dh * act(g))
enum GateMode { GATE_NONE = 0, GATE_FWD = 1, GATE_FWD_SAVE = 2, GATE_BWD = 3 };

// As ExpertArgs, with M the width of h: GATE_FWD's weights have 2 M features,
// those of the other projection `up` elements after the gate's.  out is h, or
// dgu (GATE_BWD).
struct GatedArgs : ExpertArgs {
  void* gu;       // saved (GATE_FWD_SAVE) or read (GATE_BWD): [T][2 M]
  int64_t ldgu;   // elements between its rows
  int64_t up;
  int32_t act;    // cbd_activation
};

int launch_gated_generic(const GatedArgs& a, const ExpertLaunch& l, int mode, void* stream);
int launch_gated_stream(const GatedArgs& a, const ExpertLaunch& l, int mode, void* stream);
int launch_gated_mfma(const GatedArgs& a, const ExpertLaunch& l, int mode, void* stream);
int launch_gated_mfma_bwd(const GatedArgs& a, const ExpertLaunch& l, void* stream);

}  // namespace cbd
