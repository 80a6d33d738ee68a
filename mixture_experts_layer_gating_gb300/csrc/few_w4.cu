// The few-token layer for group-scaled 4-bit expert weights.
#include "few_layer.cuh"

namespace moe {
cudaError_t launch_few_w4(int group, const FewArgs& a, cudaStream_t s) {
  if (group == 32) return launch_few_kind<kStreamW4, 32>(a, s);
  if (group == 64) return launch_few_kind<kStreamW4, 64>(a, s);
  return launch_few_kind<kStreamW4, 128>(a, s);
}
}  // namespace moe
