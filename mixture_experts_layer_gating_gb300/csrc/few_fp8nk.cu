// The few-token layer for e4m3 expert weights stored [.., N, K].
#include "few_layer.cuh"

namespace moe {
cudaError_t launch_few_fp8nk(const FewArgs& a, cudaStream_t s) { return launch_few_kind<kStreamFp8Nk, 0>(a, s); }
}  // namespace moe
