// The residual's addition, the root-mean-square norm and the normed rows in e4m3
// (moe_add_rms_norm; also the first launch of moe_block).
//
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * weight
//
// Bound by memory: every row is read once and held in registers, a group of threads to a
// row, from the sum of squares to the stores.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct NormParams {
  const void *x, *residual, *weight;
  void *sum_out, *y;
  uint8_t* q;
  float* scales;
  int rows, D, group;  // group: values to a scale, 0 = the row
  int tpr_log2;        // threads to a row, 2^5 .. 2^10
  float eps;
};

// 8 consecutive values, as loaded.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* p, long long i) { w = __ldcs(static_cast<const uint4*>(p) + i); }
  __device__ __forceinline__ void load_kept(const void* p, long long i) { w = __ldg(static_cast<const uint4*>(p) + i); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, long long i, const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    static_cast<uint4*>(p)[i] = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, long long i) {
    a = __ldcs(static_cast<const float4*>(p) + 2 * i);
    b = __ldcs(static_cast<const float4*>(p) + 2 * i + 1);
  }
  __device__ __forceinline__ void load_kept(const void* p, long long i) {
    a = __ldg(static_cast<const float4*>(p) + 2 * i);
    b = __ldg(static_cast<const float4*>(p) + 2 * i + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, long long i, const float (&f)[8]) {
    static_cast<float4*>(p)[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
    static_cast<float4*>(p)[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Sum (or largest) over the threads of a row, the same bits on each; NaN stays NaN.
template <bool MAX>
__device__ __forceinline__ float combine(float a, float b) {
  if (!MAX) return a + b;
  return a > b || a != a ? a : b;  // (b NaN: the comparison is false)
}
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = combine<MAX>(v, __shfl_xor_sync(kFull, v, o));
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5, first = warp & ~(warps - 1);
  __syncthreads();  // the last reading of red
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  v = red[first];
  for (int w = 1; w < warps; ++w) v = combine<MAX>(v, red[first + w]);
  return v;
}

__device__ __forceinline__ float e4m3_scale(float largest) {
  if (largest == 0.0f) return 1.0f;
  // (an infinity or NaN gives NaN, so that the group's products are NaN)
  return isfinite(largest) ? fmaxf(__fdiv_rn(largest, 448.0f), FLT_MIN) : __int_as_float(0x7fffffff);
}

// VPT vectors of 8 values a thread.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const NormParams p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float red[32];
  const int tpr = 1 << p.tpr_log2, rpb = blockDim.x >> p.tpr_log2;
  const int li = threadIdx.x & (tpr - 1), warps = tpr >> 5;
  const int nvec = p.D / 8;
  // (rows of several warps have a block of their own, whose threads all run the same
  // iterations and branches on the row: row_reduce's barriers)
  for (long long r0 = static_cast<long long>(blockIdx.x) * rpb; r0 < p.rows;
       r0 += static_cast<long long>(gridDim.x) * rpb) {
    const long long r = r0 + (threadIdx.x >> p.tpr_log2);
    const bool valid = r < p.rows;
    const long long base = r * nvec;
    float f[VPT][8];
    {
      Vec8<T> a[VPT], b[VPT];
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = li + tpr * j;
        if (valid && v < nvec) {
          a[j].load(p.x, base + v);
          if (p.residual) b[j].load(p.residual, base + v);
        }
      }
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (valid && li + tpr * j < nvec) {
          a[j].get(f[j]);
          if (p.residual) {
            float g[8];
            b[j].get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[j][i] += g[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[j][i] = 0.0f;
        }
      }
    }
    if (p.sum_out) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (valid && li + tpr * j < nvec) Vec8<T>::store(p.sum_out, base + li + tpr * j, f[j]);
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[j][i], f[j][i], ss);
    ss = row_reduce<false>(ss, red, warps);
    float rstd = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
    // squares that leave fp32's range (above; or below, where eps does not cover them): the
    // row times the power of two that brings its largest value to [1, 2), or, below, as far
    // as eps times its square stays in range
    if (!(ss <= 1e37f) || (ss < 1e-27f && p.eps < 1e-25f)) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = combine<true>(m, fabsf(f[j][i]));
      m = row_reduce<true>(m, red, warps);
      if (m > 0.0f && isfinite(m)) {
        const int e = max(ilogbf(m), p.eps > 0.0f ? -44 : -200);
        ss = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[j][i] = ldexpf(f[j][i], -e);
            ss = fmaf(f[j][i], f[j][i], ss);
          }
        ss = row_reduce<false>(ss, red, warps);
        rstd = rsqrtf(ss / static_cast<float>(p.D) + ldexpf(p.eps, -2 * e));
      }
    }
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = li + tpr * j;
      if (v < nvec) {
        Vec8<T> w;
        w.load_kept(p.weight, v);
        float g[8];
        w.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[j][i] = f[j][i] * rstd * g[i];
          most = combine<true>(most, fabsf(f[j][i]));
        }
        if (valid && p.y) Vec8<T>::store(p.y, base + v, f[j]);
      }
    }
    if (!p.q) continue;
    if (!p.group) {
      const float s = e4m3_scale(row_reduce<true>(most, red, warps));
      if (valid && li == 0) p.scales[r] = s;
      most = s;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = li + tpr * j;
      float s = most;
      if (p.group) {
        // group / 8 neighbouring threads hold a group (D is a multiple of it, so they
        // hold it whole or not at all)
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = combine<true>(s, fabsf(f[j][i]));
        for (int o = 1; o < p.group / 8; o <<= 1) s = combine<true>(s, __shfl_xor_sync(kFull, s, o));
        s = e4m3_scale(s);
        if (valid && v < nvec && v % (p.group / 8) == 0)
          p.scales[r * (p.D / p.group) + v / (p.group / 8)] = s;
      }
      if (valid && v < nvec) {
        const float inv = 1.0f / s;
        uint32_t u[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[i >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                           make_float2(f[j][2 * i] * inv, f[j][2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3))
                       << (16 * (i & 1));
        reinterpret_cast<uint2*>(p.q)[base + v] = make_uint2(u[0], u[1]);
      }
    }
  }
}

template <typename T, int VPT>
cudaError_t launch_vpt(const NormParams& p, cudaStream_t s) {
  const int tpr = 1 << p.tpr_log2, block = tpr == 32 ? 256 : tpr, rpb = block / tpr;
  const long long want = (static_cast<long long>(p.rows) + rpb - 1) / rpb;
  const int grid = static_cast<int>(std::min<long long>(want, 2048ll / block * device_sm_count()));
  const cudaError_t e = launch_kernel(add_rms_norm_kernel<T, VPT>, dim3(grid), dim3(block), 0, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(NormParams& p, cudaStream_t s) {
  const int nvec = p.D / 8;
  int tl = 5;
  while ((4 << tl) < nvec) ++tl;
  p.tpr_log2 = tl;
  return launch_vpt<T, 4>(p, s);
}

}  // namespace

cudaError_t launch_add_rms_norm(int rows, int D, bool f32, const void* x, const void* residual, const void* weight,
                                float eps, void* sum_out, void* y, void* q, int group, float* scales,
                                cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  NormParams p{x, residual, weight, sum_out, y, static_cast<uint8_t*>(q), scales, rows, D, group, 0, eps};
  return f32 ? launch_type<float>(p, s) : launch_type<__nv_bfloat16>(p, s);
}

}  // namespace moe
