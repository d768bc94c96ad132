// kern_gated_stream.hip -- gated experts with few rows an expert, bf16 (expert_stream.h).
#include "expert_stream.h"

namespace cbd {

int launch_gated_stream(const GatedArgs& a, const ExpertLaunch& l, int mode, void* stream) {
  const bool ak = l.form == EXPERT_AK;
  const void* k = mode == GATE_FWD ? ak ? (const void*)&expert_stream_kernel<EXPERT_AK, GATE_FWD>
                                        : (const void*)&expert_stream_kernel<EXPERT_AM, GATE_FWD>
                  : ak ? (const void*)&expert_stream_kernel<EXPERT_AK, GATE_FWD_SAVE>
                       : (const void*)&expert_stream_kernel<EXPERT_AM, GATE_FWD_SAVE>;
  void* args[] = {const_cast<GatedArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
