// kern_gated_mfma_bwd.hip -- the backward product of gated experts with many rows, bf16 (expert_mfma.h).
#include "expert_mfma.h"

namespace cbd {
namespace {

template <int FORM>
const void* pick(const GatedArgs& a, const ExpertLaunch& l) {
  if (l.bn == 256) return (const void*)&expert_mfma_kernel<uint16_t, FORM, 4, 4, true, WHOLE, GATE_BWD>;
  if (l.dma && a.whole_out) return (const void*)&expert_mfma_kernel<uint16_t, FORM, 2, 2, true, WHOLE, GATE_BWD>;
  return l.dma ? (const void*)&expert_mfma_kernel<uint16_t, FORM, 2, 2, true, ANY, GATE_BWD>
               : (const void*)&expert_mfma_kernel<uint16_t, FORM, 2, 2, false, ANY, GATE_BWD>;
}

}  // namespace

int launch_gated_mfma_bwd(const GatedArgs& a, const ExpertLaunch& l, void* stream) {
  const void* k = l.form == EXPERT_AK ? pick<EXPERT_AK>(a, l) : pick<EXPERT_AM>(a, l);
  void* args[] = {const_cast<GatedArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
