// kern_gated_mfma.hip -- gated experts with many rows, bf16 (expert_mfma.h).
#include "expert_mfma.h"

namespace cbd {
namespace {

template <int FORM, int GATE>
const void* pick(const GatedArgs& a, const ExpertLaunch& l) {
  if (l.bn == 256) return (const void*)&expert_mfma_kernel<uint16_t, FORM, 4, 4, true, WHOLE, GATE>;
  if (l.dma && a.whole_out) return (const void*)&expert_mfma_kernel<uint16_t, FORM, 2, 2, true, WHOLE, GATE>;
  return l.dma ? (const void*)&expert_mfma_kernel<uint16_t, FORM, 2, 2, true, ANY, GATE>
               : (const void*)&expert_mfma_kernel<uint16_t, FORM, 2, 2, false, ANY, GATE>;
}

}  // namespace

int launch_gated_mfma(const GatedArgs& a, const ExpertLaunch& l, int mode, void* stream) {
  if (mode == GATE_BWD) return launch_gated_mfma_bwd(a, l, stream);
  const void* k = l.form == EXPERT_AK ? mode == GATE_FWD ? pick<EXPERT_AK, GATE_FWD>(a, l) : pick<EXPERT_AK, GATE_FWD_SAVE>(a, l)
                  : mode == GATE_FWD  ? pick<EXPERT_AM, GATE_FWD>(a, l)
                                      : pick<EXPERT_AM, GATE_FWD_SAVE>(a, l);
  void* args[] = {const_cast<GatedArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
