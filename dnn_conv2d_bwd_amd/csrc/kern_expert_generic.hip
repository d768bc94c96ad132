// kern_expert_generic.hip -- expert products of any type, size, stride and alignment (expert_generic.h).
#include "expert_generic.h"

namespace cbd {
namespace {

template <typename T, typename TO, int FORM>
const void* pick(int bm) {
  return bm == 128 ? (const void*)&expert_generic_kernel<T, TO, FORM, 4>
                   : (const void*)&expert_generic_kernel<T, TO, FORM, 2>;
}

}  // namespace

int launch_expert_generic(const ExpertArgs& a, const ExpertLaunch& l, void* stream) {
  const void* k;
  if (l.form == EXPERT_DW)
    k = l.dtype == CBD_F32        ? pick<float, float, EXPERT_DW>(l.bm)
        : l.out_dtype == CBD_F32  ? pick<uint16_t, float, EXPERT_DW>(l.bm)
                                  : pick<uint16_t, uint16_t, EXPERT_DW>(l.bm);
  else if (l.form == EXPERT_AK)
    k = l.dtype == CBD_F32 ? pick<float, float, EXPERT_AK>(l.bm) : pick<uint16_t, uint16_t, EXPERT_AK>(l.bm);
  else
    k = l.dtype == CBD_F32 ? pick<float, float, EXPERT_AM>(l.bm) : pick<uint16_t, uint16_t, EXPERT_AM>(l.bm);
  void* args[] = {const_cast<ExpertArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
