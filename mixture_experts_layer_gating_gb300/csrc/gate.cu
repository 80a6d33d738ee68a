// Routing by scores, bias and groups from router logits (moe_route_gated): one warp per
// token (gate_warp.cuh).
#include <cuda_runtime.h>

#include <algorithm>

#include "gate_warp.cuh"

namespace moe {
namespace {

// v = or (ADD) += a plane's row of logits (EPL neighbouring experts of this lane; 0 past E).
template <int EPL, bool ADD>
__device__ __forceinline__ void load_logits(const float* __restrict__ row, int lane, int E, bool vec, float (&v)[EPL]) {
  const int e0 = lane * EPL;
  if (vec) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      const float4 f = e0 + i < E ? *reinterpret_cast<const float4*>(row + e0 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[i] = ADD ? v[i] + f.x : f.x;
      v[i + 1] = ADD ? v[i + 1] + f.y : f.y;
      v[i + 2] = ADD ? v[i + 2] + f.z : f.z;
      v[i + 3] = ADD ? v[i + 3] + f.w : f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float f = e0 + i < E ? row[e0 + i] : 0.0f;
      v[i] = ADD ? v[i] + f : f;
    }
  }
}

constexpr int kGateWarps = 8;

template <int EPL, bool WHOLE, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kGateWarps * 32)
    gate_kernel(const float* __restrict__ planes, int nsplit, const float* __restrict__ logit_bias,
                const float* __restrict__ select_bias, float* logits, int T, bool vec, const GateParams g,
                int32_t* __restrict__ ids, float* __restrict__ w, int32_t* err) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ __align__(16) uint32_t scratch[kGateWarps][gate_scratch(EPL)];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = static_cast<long long>(blockIdx.x) * kGateWarps + warp;
  if (t >= T) return;
  float v[EPL];
  const size_t at = static_cast<size_t>(t) * g.E;
  load_logits<EPL, false>(planes + at, lane, g.E, vec, v);
  for (int s = 1; s < nsplit; ++s)
    load_logits<EPL, true>(planes + s * (static_cast<size_t>(T) * g.E) + at, lane, g.E, vec, v);
  warp_gate_topk<EPL, WHOLE, SIGMOID, BIAS>(v, lane, g, logit_bias, select_bias,
                                            (nsplit > 1 || logit_bias) ? logits + at : nullptr, ids + t * g.k,
                                            w + t * g.k, scratch[warp], err);
}

template <int EPL, bool WHOLE>
auto gate_kernel_of(bool sigmoid, bool bias) {
  return sigmoid ? (bias ? gate_kernel<EPL, WHOLE, true, true> : gate_kernel<EPL, WHOLE, true, false>)
                 : (bias ? gate_kernel<EPL, WHOLE, false, true> : gate_kernel<EPL, WHOLE, false, false>);
}

}  // namespace

cudaError_t launch_gate(const float* planes, int nsplit, const float* logit_bias, const float* select_bias,
                        float* logits, int T, const GateParams& g, int32_t* ids, float* w, int32_t* err,
                        cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  const int blocks = (T + kGateWarps - 1) / kGateWarps;
  const bool vec = g.E % 4 == 0 && !(reinterpret_cast<uintptr_t>(planes) & 15);
  const bool sg = g.sigmoid, sb = select_bias != nullptr;
  auto kern = g.E <= 128   ? (g.E % 4 ? gate_kernel_of<4, false>(sg, sb) : gate_kernel_of<4, true>(sg, sb))
              : g.E <= 256 ? (g.E % 8 ? gate_kernel_of<8, false>(sg, sb) : gate_kernel_of<8, true>(sg, sb))
                           : (g.E % 16 ? gate_kernel_of<16, false>(sg, sb) : gate_kernel_of<16, true>(sg, sb));
  const cudaError_t e = launch_kernel(kern, dim3(blocks), dim3(kGateWarps * 32), 0, s, planes, nsplit, logit_bias,
                                      select_bias, logits, T, vec, g, ids, w, err);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
