// C ABI of the operators for a few tokens (include/moe.h): moe_layer_few,
// moe_linear_w4, moe_quantize_w4, moe_dequantize_w4.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "few_layer.cuh"

using namespace moe;

namespace {

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The layout-dependent widths of the kernel for a weight type (StreamTraits).
struct FewGeom {
  int kch, hc;
};
FewGeom few_geom(int w_dtype) {
  switch (w_dtype) {
    case MOE_BF16: return {StreamTraits<kStreamBf16, 0>::KCH, StreamTraits<kStreamBf16, 0>::HC};
    case MOE_FP8_E4M3: return {StreamTraits<kStreamFp8, 0>::KCH, StreamTraits<kStreamFp8, 0>::HC};
    case MOE_FP8_E4M3_NK: return {StreamTraits<kStreamFp8Nk, 0>::KCH, StreamTraits<kStreamFp8Nk, 0>::HC};
    default: return {StreamTraits<kStreamW4, 32>::KCH, StreamTraits<kStreamW4, 32>::HC};
  }
}

bool few_dtype(const moe_config_t* c) {
  return c->act_dtype == MOE_BF16 && (c->w_dtype == MOE_BF16 || c->w_dtype == MOE_FP8_E4M3 ||
                                      c->w_dtype == MOE_FP8_E4M3_NK || w4_group(c->w_dtype));
}

int few_planes(const moe_config_t* c) {
  // at least two k16 steps per warp of a unit, at most one unit per CTA of a GB300's
  // 152 (a constant: the workspace's size must not depend on the current device)
  const int steps = ceil_div(c->D, 16), se = ceil_div(c->E, 64);
  return std::max(1, std::min({kFewMaxPlanes, steps / 16, 152 / se}));
}

struct FewLayout {
  size_t cnt, planes, xp, xinv, hp, hmax, part, prim, extra, total;
  int Dp, Ip, W;
};
FewLayout few_layout(const moe_config_t* c) {
  const FewGeom g = few_geom(c->w_dtype);
  FewLayout L{};
  L.Dp = ceil_div(c->D, g.kch) * g.kch;
  L.Ip = ceil_div(std::max(c->I, c->I_shared), g.kch) * g.kch;
  L.W = 2 * g.hc * ceil_div(c->D, 2 * g.hc);
  const size_t T = c->T, rows = T * c->k + T;
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur = up256(cur + bytes);
    return o;
  };
  L.cnt = take(kStreamMaxCtas * 4);
  L.planes = take(static_cast<size_t>(few_planes(c)) * T * c->E * 4);
  L.xp = take(T * L.Dp * 2);
  L.xinv = take(T * 4);
  L.hp = take(rows * L.Ip * 4);
  L.hmax = take(rows * 4);
  L.part = take(static_cast<size_t>(2) * kStreamMaxCtas * T * 2 * g.hc * 4);
  L.prim = take(rows * L.W * 4);
  L.extra = take(static_cast<size_t>(kStreamMaxCtas) * T * 2 * g.hc * 4);
  L.total = cur;
  return L;
}

constexpr int kW4MaxN = 0x7ffffe00;  // whole strips of columns stay below 2^31
bool w4_args_ok(int64_t G, int K, int N, int group) {
  return G >= 1 && G <= 65535 && (group == 32 || group == 64 || group == 128) && K >= group &&
         K % group == 0 && K / group <= 65535 && N >= 1 && N <= kW4MaxN;
}

}  // namespace

namespace moe {

size_t few_workspace_bytes(const moe_config_t* c) {
  return few_dtype(c) && c->T >= 1 && c->T <= kStreamMaxRows ? few_layout(c).total : 0;
}

}  // namespace moe

extern "C" {

int moe_layer_few(const moe_config_t* cfg, const void* x, const void* Wg, const float* logit_bias,
                  const void* W13, const void* s13, const void* W2, const void* s2, const void* W13s,
                  const void* s13s, const void* W2s, const void* s2s, void* out, void* ws,
                  size_t ws_bytes, void* stream) {
  if (!cfg_valid(cfg)) return MOE_ERR_INVALID_ARG;
  if (!few_dtype(cfg) || cfg->T > kStreamMaxRows) return MOE_ERR_UNSUPPORTED;
  const size_t need = moe_workspace_size(cfg);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < need) return MOE_ERR_WORKSPACE;
  for (const void* q : {x, Wg, W13, W2, static_cast<const void*>(out)})
    if (!q || !al16(q)) return MOE_ERR_INVALID_ARG;
  const bool scaled = cfg->w_dtype != MOE_BF16, shared = cfg->I_shared > 0;
  if (scaled != (s13 != nullptr) || scaled != (s2 != nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {s13, s2, shared ? s13s : nullptr, shared ? s2s : nullptr})
    if (!al16(q)) return MOE_ERR_INVALID_ARG;
  if (shared) {
    if (!W13s || !W2s || !al16(W13s) || !al16(W2s)) return MOE_ERR_INVALID_ARG;
    if (scaled != (s13s != nullptr) || scaled != (s2s != nullptr)) return MOE_ERR_INVALID_ARG;
  }
  if (cfg->T == 0) return MOE_OK;
  const FewLayout L = few_layout(cfg);
  uint8_t* base = static_cast<uint8_t*>(ws);
  uint8_t* few = base + (need - L.total);  // the last region of the workspace
  FewArgs a{};
  FewParams& p = a.p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.Wg = static_cast<const __nv_bfloat16*>(Wg);
  p.bias = logit_bias;
  p.s13 = s13;
  p.s2 = s2;
  p.s13s = s13s;
  p.s2s = s2s;
  p.out = static_cast<__nv_bfloat16*>(out);
  ControlBlock* cb = reinterpret_cast<ControlBlock*>(ws);
  p.err = &cb->err;
  p.bar = reinterpret_cast<uint32_t*>(cb->reserved + kGridBarrierSlot);
  p.cnt = reinterpret_cast<int32_t*>(few + L.cnt);
  p.logits = reinterpret_cast<float*>(base + moe_workspace_offset(cfg, MOE_WS_LOGITS));
  p.ids = reinterpret_cast<int32_t*>(base + moe_workspace_offset(cfg, MOE_WS_TOPK_IDS));
  p.topw = reinterpret_cast<float*>(base + moe_workspace_offset(cfg, MOE_WS_TOPK_W));
  p.planes = reinterpret_cast<float*>(few + L.planes);
  p.xp = reinterpret_cast<uint16_t*>(few + L.xp);
  p.xinv = reinterpret_cast<float*>(few + L.xinv);
  p.hp = few + L.hp;
  p.hmax = reinterpret_cast<uint32_t*>(few + L.hmax);
  p.part = reinterpret_cast<float*>(few + L.part);
  p.prim = reinterpret_cast<float*>(few + L.prim);
  p.extra = reinterpret_cast<float*>(few + L.extra);
  p.T = cfg->T;
  p.D = cfg->D;
  p.E = cfg->E;
  p.k = cfg->k;
  p.I = cfg->I;
  p.Is = cfg->I_shared;
  p.act = cfg->act;
  p.renorm = cfg->renormalize;
  p.Dp = L.Dp;
  p.Ip = L.Ip;
  p.W = L.W;
  p.nplanes = few_planes(cfg);
  a.W13 = W13;
  a.W2 = W2;
  a.W13s = W13s;
  a.W2s = W2s;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (cfg->w_dtype) {
    case MOE_BF16: e = launch_few_bf16(a, s); break;
    case MOE_FP8_E4M3: e = launch_few_fp8(a, s); break;
    case MOE_FP8_E4M3_NK: e = launch_few_fp8nk(a, s); break;
    default: e = launch_few_w4(w4_group(cfg->w_dtype), a, s); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_linear_w4_workspace_size(int32_t M, int32_t K, int32_t N) {
  if (M < 0 || M > kStreamMaxRows || K < 32 || K % 32 || N < 1 || N > kW4MaxN) return 0;
  return sizeof(ControlBlock) + linear_w4_scratch(std::max(M, 1), K, N).total;
}

int moe_linear_w4(int32_t M, int32_t K, int32_t N, int32_t group, const void* x, const void* Wq,
                  const void* scales, const void* zeros, void* y, int32_t y_dtype, void* ws,
                  size_t ws_bytes, void* stream) {
  if (M < 0 || !w4_args_ok(1, K, N, group)) return MOE_ERR_INVALID_ARG;
  if (M > kStreamMaxRows || (y_dtype != MOE_BF16 && y_dtype != MOE_F32)) return MOE_ERR_UNSUPPORTED;
  const size_t need = moe_linear_w4_workspace_size(M, K, N);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (M == 0) return MOE_OK;  // (an empty x or y may have no address)
  for (const void* q : {x, Wq, scales, static_cast<const void*>(y)})
    if (!q || !al16(q)) return MOE_ERR_INVALID_ARG;
  const cudaError_t e =
      launch_linear_w4(M, K, N, group, x, Wq, scales, static_cast<const uint8_t*>(zeros), y,
                       y_dtype == MOE_F32, &reinterpret_cast<ControlBlock*>(ws)->err,
                       static_cast<uint8_t*>(ws) + sizeof(ControlBlock), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_quantize_w4(const void* W, int32_t w_dtype, int64_t G, int32_t K, int32_t N, int32_t group,
                    void* Wq, void* scales, void* stream) {
  if (!W || !Wq || !scales || !al16(W) || !al16(Wq) || !al16(scales) || !w4_args_ok(G, K, N, group))
    return MOE_ERR_INVALID_ARG;
  if (w_dtype != MOE_BF16 && w_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  const cudaError_t e = launch_quantize_w4(W, w_dtype == MOE_F32, G, K, N, group, Wq, scales,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_dequantize_w4(const void* Wq, const void* scales, const void* zeros, int64_t G, int32_t K,
                      int32_t N, int32_t group, void* W, void* stream) {
  if (!W || !Wq || !scales || !al16(W) || !al16(Wq) || !al16(scales) || !w4_args_ok(G, K, N, group))
    return MOE_ERR_INVALID_ARG;
  const cudaError_t e = launch_dequantize_w4(Wq, scales, static_cast<const uint8_t*>(zeros), G, K, N, group,
                                             W, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
