// The residual's addition, the root-mean-square norm and the normed rows in e4m3
// (moe_add_rms_norm; also the first launch of moe_block).
//
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * weight
//
// Bound by memory: every row is read once and held in registers, a group of threads to a
// row, from the sum of squares to the stores.  Measured (one GB300, inputs rotated so that
// they come from HBM; share of what a copy reaches): 16384 x 8192 bf16 with residual, sum, y
// and e4m3 rows 193 us (6.3 TB/s, 0.92), 8192 x 4096 the same 51 us (0.86), 4096 x 2048 fp32
// 13.6 us (0.73: launch and first bytes are 3 of them), one row of 2048 1.5 us.  Four vectors
// of 8 values a thread and 16 warps an SM: with two vectors and more warps 206 us, 67 us, 15.1
// us; with the row read again for the norm it would move a third more.  Farther from a copy:
// 2000 x 4096 with scales of 128 17.2 us (0.62: 608 blocks take 3.3 rows each), and rows of more
// than 16384 values, whose eight vectors a thread spill registers and leave none for the next
// row (4096 x 32768 bf16 with row scales 285 us, 0.62; fp32 without 521 us, 0.61).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxTprLog2 = 9, kMaxWarps = 1 << (kMaxTprLog2 - 5);  // threads to a row, 2^5 .. 2^9
constexpr int kSms = 152;  // a constant, for the choice of threads to a row: results must not depend on the device

struct NormParams {
  const void *x, *residual, *weight;
  void *sum_out, *y;
  uint8_t* q;
  float* scales;
  int rows, D, group;  // group: values to a scale, 0 = the row
  int tpr_log2;        // threads to a row
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

// Sum over the threads of a row, or the largest of unsigned numbers, the same on each.
// Magnitudes are compared as the unsigned bits of |f|, which order as they do and put NaN
// above infinity.
__device__ __forceinline__ float join(float a, float b) { return a + b; }
__device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return max(a, b); }
template <typename V>
__device__ __forceinline__ V row_reduce(V v, V* red, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(kFull, v, o));
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? red[lane] : V(0);
#pragma unroll
  for (int o = kMaxWarps / 2; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(kFull, v, o));
  return __shfl_sync(kFull, v, 0);
}
__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

__device__ __forceinline__ float e4m3_scale(uint32_t largest) {
  if (largest == 0u) return 1.0f;
  // (an infinity or NaN gives NaN, so that the group's products are NaN)
  return largest < 0x7f800000u ? fmaxf(__fdiv_rn(__uint_as_float(largest), 448.0f), FLT_MIN)
                               : __uint_as_float(0x7fffffffu);
}
// Two fp32 values to a register pair, for the instructions that take both at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// e4m3 of the fp32 quotients f / scale, rounded to nearest; inv: 1 / scale, rounded.  The
// product with the inverse is within two ulps of the quotient, one correction by its remainder
// brings it within one, and the next, whose remainder is exact, rounds as division does
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990).  Without them a quotient next to the middle of two codes takes the wrong one, 9 of a
// million; by __fdiv_rn 16384 x 8192 take 209 us, not 192.  Two values at a time, and minus the
// quotient, which keeps the sign of a zero.
__device__ __forceinline__ uint2 e4m3_codes(const float (&f)[8], float scale, float inv) {
  uint64_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
  if (scale < 0x1p-60f) {  // times 2^64, exactly: no remainder is subnormal
    scale *= 0x1p64f;
    inv *= 0x1p-64f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], pair(0x1p64f, 0x1p64f));
  }
  const uint64_t by = pair(scale, scale), minus = pair(-inv, -inv);
  uint32_t u[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t q = mul2(v[i], minus);
    q = fma2(fma2(q, by, v[i]), minus, q);
    q = fma2(fma2(q, by, v[i]), minus, q);
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(q));
    u[i >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3)) << (16 * (i & 1));
  }
  return make_uint2(u[0] ^ 0x80808080u, u[1] ^ 0x80808080u);
}

enum QMode { kNoQ, kRowQ, kGroupQ };

// VPT vectors of 8 values a thread.  Each block takes rows in turn (a row of one warp: a
// block takes eight).  Where registers allow, it has the next row's loads under way while it
// reduces and stores this one's, and keeps its part of the weight.
template <typename T, int VPT, bool ADD, QMode Q>
__global__ void __launch_bounds__(32 * kMaxWarps) add_rms_norm_kernel(const NormParams p) {
  pdl_wait();
  pdl_launch_dependents();
  // two of each, taken in turn: one barrier a reduction (the next use of the same is
  // behind the other's barrier)
  __shared__ float red[2][kMaxWarps];
  __shared__ uint32_t redm[2][kMaxWarps];
  const int tpr = 1 << p.tpr_log2, rpb = blockDim.x >> p.tpr_log2;
  const int li = threadIdx.x & (tpr - 1), warps = tpr >> 5;
  const int nvec = p.D / 8;
  const float rD = 1.0f / static_cast<float>(p.D);
  constexpr bool kAhead = VPT <= 4, kKeep = VPT * sizeof(T) <= 8;
  Vec8<T> a[VPT], b[VPT], w[VPT];
  auto load = [&](long long r) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = li + tpr * j;
      if (r < p.rows && v < nvec) {
        a[j].load(p.x, r * nvec + v);
        if (ADD) b[j].load(p.residual, r * nvec + v);
      }
    }
  };
  long long r = static_cast<long long>(blockIdx.x) * rpb + (threadIdx.x >> p.tpr_log2);
  const long long step = static_cast<long long>(gridDim.x) * rpb;
  load(r);
  if (kKeep) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (li + tpr * j < nvec) w[j].load_kept(p.weight, li + tpr * j);
  }
  // (rows of several warps have a block of their own, whose threads all run the same
  // iterations and branches on the row: row_reduce's barriers)
  for (int buf = 0; r < p.rows; r += step, buf ^= 1) {
    const long long base = r * nvec;
    float f[VPT][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (li + tpr * j < nvec) {
        a[j].get(f[j]);
        if (ADD) {
          float g[8];
          b[j].get(g);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[j][i] += g[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j][i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[j][i], f[j][i], ss);
    }
    if (kAhead) load(r + step);
    if (p.sum_out) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (li + tpr * j < nvec) Vec8<T>::store(p.sum_out, base + li + tpr * j, f[j]);
    }
    ss = row_reduce(ss, red[buf], warps);
    float rstd = rsqrtf(fmaf(ss, rD, p.eps));
    // squares that leave fp32's range (above; or below, where eps does not cover them): the
    // row times the power of two that brings its largest value to [1, 2), or, below, as far
    // as eps times its square stays in range
    if (!(ss <= 1e37f) || (ss < 1e-27f && p.eps < 1e-25f)) {
      uint32_t m = 0u;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, magnitude(f[j][i]));
      if (warps > 1) __syncthreads();
      m = row_reduce(m, redm[buf], warps);
      if (m > 0u && m < 0x7f800000u) {
        const int e = max(ilogbf(__uint_as_float(m)), p.eps > 0.0f ? -44 : -200);
        ss = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[j][i] = ldexpf(f[j][i], -e);
            ss = fmaf(f[j][i], f[j][i], ss);
          }
        ss = row_reduce(ss, red[buf], warps);
        rstd = rsqrtf(fmaf(ss, rD, ldexpf(p.eps, -2 * e)));
      }
      if (warps > 1) __syncthreads();
    }
    uint32_t most[VPT];
    uint32_t all = 0u;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      most[j] = 0u;
      if (li + tpr * j < nvec) {
        float g[8];
        if (!kKeep) w[j].load_kept(p.weight, li + tpr * j);
        w[j].get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[j][i] = f[j][i] * rstd * g[i];
          if (Q != kNoQ) most[j] = max(most[j], magnitude(f[j][i]));
        }
        if (p.y) Vec8<T>::store(p.y, base + li + tpr * j, f[j]);
      }
      all = max(all, most[j]);
    }
    if (Q == kRowQ) {
      const float s = e4m3_scale(row_reduce(all, redm[buf], warps));
      if (li == 0) p.scales[r] = s;
      const float inv = __frcp_rn(s);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (li + tpr * j < nvec) reinterpret_cast<uint2*>(p.q)[base + li + tpr * j] = e4m3_codes(f[j], s, inv);
    }
    if (Q == kGroupQ) {
      // group / 8 neighbouring threads hold a group (D is a multiple of it, so they hold it
      // whole or not at all)
      const int lanes = p.group / 8;
      // scales and their inverses: those of four vectors by a lane each (four neighbours are
      // of one group)
      constexpr int C = VPT < 4 ? 1 : 4;
#pragma unroll
      for (int j0 = 0; j0 < VPT; j0 += C) {
        uint32_t mine = 0u;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          uint32_t m = most[j0 + c];
          for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
          if (C == 1 || (li & 3) == c) mine = m;
        }
        const float my_s = e4m3_scale(mine), my_inv = __frcp_rn(my_s);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float s = C == 1 ? my_s : __shfl_sync(kFull, my_s, c, 4);
          const float inv = C == 1 ? my_inv : __shfl_sync(kFull, my_inv, c, 4);
          const int v = li + tpr * (j0 + c);
          if (v < nvec) {
            if (v % lanes == 0) p.scales[r * (nvec / lanes) + v / lanes] = s;
            reinterpret_cast<uint2*>(p.q)[base + v] = e4m3_codes(f[j0 + c], s, inv);
          }
        }
      }
    }
    if (!kAhead) load(r + step);
  }
}

template <typename T, int VPT, bool ADD>
cudaError_t launch_q(const NormParams& p, cudaStream_t s) {
  auto kern = !p.q ? add_rms_norm_kernel<T, VPT, ADD, kNoQ>
                   : p.group ? add_rms_norm_kernel<T, VPT, ADD, kGroupQ> : add_rms_norm_kernel<T, VPT, ADD, kRowQ>;
  const int tpr = 1 << p.tpr_log2, block = tpr == 32 ? 256 : tpr, rpb = block / tpr;
  const long long want = (static_cast<long long>(p.rows) + rpb - 1) / rpb;
  // (as many as 512 threads an SM: what their registers allow)
  const int grid = static_cast<int>(std::min<long long>(want, 512ll / block * device_sm_count()));
  const cudaError_t e = launch_kernel(kern, dim3(grid), dim3(block), 0, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename T, int VPT>
cudaError_t launch_vpt(const NormParams& p, cudaStream_t s) {
  return p.residual ? launch_q<T, VPT, true>(p, s) : launch_q<T, VPT, false>(p, s);
}

template <typename T>
cudaError_t launch_type(NormParams& p, cudaStream_t s) {
  const int nvec = p.D / 8;
  auto threads = [&](int vpt) {
    int tl = 5;
    while ((vpt << tl) < nvec) ++tl;
    return tl;
  };
  // few rows (one or two to an SM): every thread has one vector, for the shortest chain
  if (p.rows <= 2 * kSms && threads(1) <= kMaxTprLog2) {
    p.tpr_log2 = threads(1);
    return launch_vpt<T, 1>(p, s);
  }
  if (threads(4) <= kMaxTprLog2) {
    p.tpr_log2 = threads(4);
    return launch_vpt<T, 4>(p, s);
  }
  p.tpr_log2 = threads(8);
  return launch_vpt<T, 8>(p, s);
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
