// kern_expert_stream.hip -- bf16 expert products with few rows an expert (expert_stream.h).
#include "expert_stream.h"

namespace cbd {
int launch_expert_stream(const ExpertArgs& a, const ExpertLaunch& l, void* stream) {
  const void* k = l.form == EXPERT_AK ? (const void*)&expert_stream_kernel<EXPERT_AK>
                                      : (const void*)&expert_stream_kernel<EXPERT_AM>;
  void* args[] = {const_cast<ExpertArgs*>(&a)};
  return (int)hipLaunchKernel(k, dim3((unsigned)l.grid), dim3(THREADS), args, 0, (hipStream_t)stream);
}

}  // namespace cbd
