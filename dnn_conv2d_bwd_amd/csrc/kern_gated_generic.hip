// kern_gated_generic.hip -- gated experts of any type, size, stride and alignment (expert_generic.h).
#include "expert_generic.h"

namespace cbd {
namespace {

template <typename T, int FORM, int GATE>
const void* pick(int bm) {
  return bm == 128 ? (const void*)&expert_generic_kernel<T, T, FORM, 4, GATE>
                   : (const void*)&expert_generic_kernel<T, T, FORM, 2, GATE>;
}
template <typename T, int FORM>
const void* pick(int bm, int mode) {
  return mode == GATE_FWD        ? pick<T, FORM, GATE_FWD>(bm)
         : mode == GATE_FWD_SAVE ? pick<T, FORM, GATE_FWD_SAVE>(bm)
                                 : pick<T, FORM, GATE_BWD>(bm);
}

}  // namespace

int launch_gated_generic(const GatedArgs& a, const ExpertLaunch& l, int mode, void* stream) {
  const bool f32 = l.dtype == CBD_F32;
  const void* k = l.form == EXPERT_AK ? f32 ? pick<float, EXPERT_AK>(l.bn, mode) : pick<uint16_t, EXPERT_AK>(l.bn, mode)
                  : f32               ? pick<float, EXPERT_AM>(l.bn, mode)
                                      : pick<uint16_t, EXPERT_AM>(l.bn, mode);
  void* args[] = {const_cast<GatedArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
