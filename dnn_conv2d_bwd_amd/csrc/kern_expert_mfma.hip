// kern_expert_mfma.hip -- bf16 expert products with many rows (expert_mfma.h).
#include "expert_mfma.h"

namespace cbd {
namespace {

template <typename TO, int FORM>
const void* pick(const ExpertArgs& a, const ExpertLaunch& l) {
  if (l.bn == 256) {  // with dma and whole_out
    if constexpr (FORM == EXPERT_DW)
      if (a.accumulate) return (const void*)&expert_mfma_kernel<TO, FORM, 4, 4, true, WHOLE_ADD>;
    return (const void*)&expert_mfma_kernel<TO, FORM, 4, 4, true, WHOLE>;
  }
  if (l.dma && a.whole_out && !a.accumulate) return (const void*)&expert_mfma_kernel<TO, FORM, 2, 2, true, WHOLE>;
  return l.dma ? (const void*)&expert_mfma_kernel<TO, FORM, 2, 2, true, ANY>
               : (const void*)&expert_mfma_kernel<TO, FORM, 2, 2, false, ANY>;
}

}  // namespace

int launch_expert_mfma(const ExpertArgs& a, const ExpertLaunch& l, void* stream) {
  const void* k = l.form == EXPERT_AK   ? pick<uint16_t, EXPERT_AK>(a, l)
                  : l.form == EXPERT_AM ? pick<uint16_t, EXPERT_AM>(a, l)
                  : l.out_dtype == CBD_F32 ? pick<float, EXPERT_DW>(a, l)
                                           : pick<uint16_t, EXPERT_DW>(a, l);
  void* args[] = {const_cast<ExpertArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
