// C ABI of the operators around the experts that need no configuration (include/moe.h):
// moe_add_rms_norm, moe_lora; and moe_call.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "moe_internal.h"

using namespace moe;

namespace {

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool width_ok(int v) { return v >= 8 && v % 8 == 0 && v <= kLoraMaxWidth; }

// MOE_OK, or why sizes are not taken
int lora_sizes(int T, int K, int N, int r, int n) {
  if (T < 0 || T > (1 << 30) || !width_ok(K) || !width_ok(N) || r < 8 || r % 8 || n < 1) return MOE_ERR_INVALID_ARG;
  return r > kLoraMaxRank || n > kLoraMaxAdapters ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

int moe_add_rms_norm(int32_t rows, int32_t D, int32_t dtype, const void* x, const void* residual,
                     const void* weight, float eps, void* sum_out, void* y, void* q, int32_t q_group,
                     float* q_scales, void* stream) {
  if (rows < 0 || D < 8 || D % 8 || !(eps >= 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (q_group != 0 && q_group != 32 && q_group != 64 && q_group != 128) return MOE_ERR_INVALID_ARG;
  if (q_group && D % q_group) return MOE_ERR_INVALID_ARG;
  if ((dtype != MOE_BF16 && dtype != MOE_F32) || D > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;  // (empty tensors may have no address)
  if (!x || !weight || (!y && !q) || (y && sum_out == y) || (q != nullptr) != (q_scales != nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {x, residual, weight, static_cast<const void*>(sum_out), static_cast<const void*>(y),
                        static_cast<const void*>(q), static_cast<const void*>(q_scales)})
    if (!al16(p)) return MOE_ERR_INVALID_ARG;
  const cudaError_t e = launch_add_rms_norm(rows, D, dtype == MOE_F32, x, residual, weight, eps, sum_out, y, q, q_group,
                                            q_scales, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_lora_workspace_size(int32_t T, int32_t K, int32_t N, int32_t r, int32_t n) {
  return lora_sizes(T, K, N, r, n) == MOE_OK ? lora_workspace_bytes(T, K, N, r, n) : 0;
}

int moe_lora(int32_t T, int32_t K, int32_t N, int32_t r, int32_t n, const void* x, const int32_t* ids,
             const void* A, const void* B, const float* scales, const void* base, void* y, int32_t y_dtype,
             void* ws, size_t ws_bytes, void* stream) {
  const int st = lora_sizes(T, K, N, r, n);
  if (st != MOE_OK) return st;
  if (y_dtype != MOE_BF16 && y_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < lora_need_bytes(T, K, N, r, n))
    return MOE_ERR_WORKSPACE;
  if (T == 0) return MOE_OK;  // (empty tensors may have no address)
  for (const void* p : {x, A, B, static_cast<const void*>(y)})
    if (!p || !al16(p)) return MOE_ERR_INVALID_ARG;
  if (!ids || !al4(ids) || !al4(scales) || !al16(base) || y == x) return MOE_ERR_INVALID_ARG;
  const cudaError_t e = launch_lora(T, K, N, r, n, x, ids, A, B, scales, base, y, y_dtype == MOE_F32,
                                    static_cast<uint8_t*>(ws), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_call(int32_t call, const void* words) {
  if (!words) return MOE_ERR_INVALID_ARG;
  const char* at = static_cast<const char*>(words);
  auto word = [&]() {
    int64_t v;
    std::memcpy(&v, at, sizeof(v));
    at += sizeof(v);
    return v;
  };
  bool fits = true;  // no integer of more than 32 bits
  auto i32 = [&]() {
    const int64_t v = word();
    fits = fits && v == static_cast<int32_t>(v);
    return static_cast<int32_t>(v);
  };
  auto ptr = [&]() { return reinterpret_cast<void*>(word()); };
  switch (call) {
    case MOE_CALL_ADD_RMS_NORM: {
      const int32_t rows = i32(), D = i32(), dtype = i32();
      const void *x = ptr(), *residual = ptr(), *weight = ptr();
      double eps;
      std::memcpy(&eps, at, sizeof(eps));
      at += sizeof(eps);
      void *sum_out = ptr(), *y = ptr(), *q = ptr();
      const int32_t group = i32();
      float* scales = static_cast<float*>(ptr());
      if (!fits) return MOE_ERR_INVALID_ARG;
      return moe_add_rms_norm(rows, D, dtype, x, residual, weight, static_cast<float>(eps), sum_out, y, q, group,
                              scales, ptr());
    }
    case MOE_CALL_ROUTE_GATED: {
      const auto* cfg = static_cast<const moe_config_t*>(ptr());
      const auto* gate = static_cast<const moe_gate_t*>(ptr());
      const void *x = ptr(), *Wg = ptr();
      const float *lb = static_cast<const float*>(ptr()), *sb = static_cast<const float*>(ptr());
      float* logits = static_cast<float*>(ptr());
      int32_t* ids = static_cast<int32_t*>(ptr());
      float* w = static_cast<float*>(ptr());
      void* ws = ptr();
      const size_t bytes = static_cast<size_t>(word());
      return moe_route_gated(cfg, gate, x, Wg, lb, sb, logits, ids, w, ws, bytes, ptr());
    }
    case MOE_CALL_LORA: {
      const int32_t T = i32(), K = i32(), N = i32(), r = i32(), n = i32();
      const void* x = ptr();
      const int32_t* ids = static_cast<const int32_t*>(ptr());
      const void *A = ptr(), *B = ptr();
      const float* scales = static_cast<const float*>(ptr());
      const void* base = ptr();
      void* y = ptr();
      const int32_t y_dtype = i32();
      void* ws = ptr();
      const size_t bytes = static_cast<size_t>(word());
      if (!fits) return MOE_ERR_INVALID_ARG;
      return moe_lora(T, K, N, r, n, x, ids, A, B, scales, base, y, y_dtype, ws, bytes, ptr());
    }
    default: return MOE_ERR_INVALID_ARG;
  }
}

}  // extern "C"
