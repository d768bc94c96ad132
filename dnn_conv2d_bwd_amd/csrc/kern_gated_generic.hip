// kern_gated_generic.hip -- gated experts of any type, size, stride and alignment (expert_generic.h).
#include "expert_generic.h"

namespace cbd {
namespace {

template <typename T, int FORM>
const void* pick(int mode) {
  return mode == GATE_FWD        ? (const void*)&expert_generic_kernel<T, T, FORM, 2, GATE_FWD>
         : mode == GATE_FWD_SAVE ? (const void*)&expert_generic_kernel<T, T, FORM, 2, GATE_FWD_SAVE>
                                 : (const void*)&expert_generic_kernel<T, T, FORM, 2, GATE_BWD>;
}

}  // namespace

int launch_gated_generic(const GatedArgs& a, const ExpertLaunch& l, int mode, void* stream) {
  const bool f32 = l.dtype == CBD_F32;
  const void* k = l.form == EXPERT_AK ? f32 ? pick<float, EXPERT_AK>(mode) : pick<uint16_t, EXPERT_AK>(mode)
                  : f32               ? pick<float, EXPERT_AM>(mode)
                                      : pick<uint16_t, EXPERT_AM>(mode);
  void* args[] = {const_cast<GatedArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
