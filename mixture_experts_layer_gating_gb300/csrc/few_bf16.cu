// The few-token layer for bf16 expert weights.
#include "few_layer.cuh"

namespace moe {
cudaError_t launch_few_bf16(const FewArgs& a, cudaStream_t s) { return launch_few_kind<kStreamBf16, 0>(a, s); }
}  // namespace moe
