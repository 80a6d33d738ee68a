// What the two kernels of moe_linear_w4 share (linear_w4.cu, linear_w4_wide.cu).
#pragma once

#include "stream_sm103.cuh"

namespace moe {

constexpr int kLinStrip = 128;  // output features of a strip (one stage's rows)
constexpr int kWideStrip = 256; // of a strip of the kernel for many rows
// Whether a product is tcgen05's (linear_w4_wide.cu).  From 17 rows on, where
// mma.sync takes longer than HBM (32 rows x 4096 x 131072: 170 us against 74), and
// for 9 to 16 rows where a launch of its own for the order of x is small against
// the weights (16 rows: 91 against 74 us at 4096 x 131072, even at 8192 x 8192, 12.9
// against 15.5 at 2816 x 4224).
inline bool linear_w4_wide(int M, int K, int N) {
  const long long stages = (static_cast<long long>(N) + kWideStrip - 1) / kWideStrip * ((K + 255) / 256);
  return M > 16 || (M > 8 && stages >= 1024);
}

struct LinParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* sc;
  const uint8_t* zp;
  void* y;
  int32_t* err;
  int32_t* cnt;   // [ctas] arrivals, zero between launches
  float* part;    // [ctas][2][M][strip]: a CTA's part of a strip begun earlier, of one it leaves unfinished
  // many rows: x put in the weights' k order by a launch of its own
  __nv_bfloat16* xp;  // [M][Kp], Kp whole stages
  int M, K, N, Kp;
};

__device__ __forceinline__ void store_y(float* y, size_t at, float v) { y[at] = v; }
__device__ __forceinline__ void store_y(__nv_bfloat16* y, size_t at, float v) {
  y[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void store_y(float* y, size_t at, float4 v) { *reinterpret_cast<float4*>(y + at) = v; }
__device__ __forceinline__ void store_y(__nv_bfloat16* y, size_t at, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(y + at) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// A whole strip's sums (RP floats a row) to y by THREADS threads.
template <int THREADS, int STRIP, typename TY>
__device__ __forceinline__ void lin_write(const LinParams& p, const float* sums, int RP, int s, int i0) {
  TY* y = static_cast<TY*>(p.y);
  const int n0 = s * STRIP;
  if ((p.N & 3) == 0) {
#pragma unroll 4
    for (int i = i0; i < p.M * (STRIP / 4); i += THREADS) {
      const int row = i / (STRIP / 4), col = i % (STRIP / 4) * 4;
      if (n0 + col < p.N)
        store_y(y, static_cast<size_t>(row) * p.N + n0 + col, *reinterpret_cast<const float4*>(sums + row * RP + col));
    }
  } else {
#pragma unroll 4
    for (int i = i0; i < p.M * STRIP; i += THREADS) {
      const int row = i / STRIP, col = i % STRIP;
      if (n0 + col < p.N) store_y(y, static_cast<size_t>(row) * p.N + n0 + col, sums[row * RP + col]);
    }
  }
}

// One strip's sums (or this CTA's part of them) to y by THREADS threads: one warp,
// or threads that meet at bar_consumers.  A strip inside one CTA's run is written
// at once; one that several CTAs share gets its parts added, in the order of k, by
// the CTA that arrives last (a count for each CTA that begins a shared strip).
template <int THREADS, int STRIP, typename TY>
__device__ __noinline__ void lin_finish(const LinParams& p, const Split& sp, float* sums, int RP, int s, int kc,
                                        int end, int C, int b, int i0, int* flag) {
  const int items = p.M * STRIP;
  if (end == C && kc == 0) {
    lin_write<THREADS, STRIP, TY>(p, sums, RP, s, i0);
    return;
  }
  float* mine = p.part + (static_cast<size_t>(b) * 2 + (kc ? 0 : 1)) * items;
#pragma unroll 4
  for (int i = i0 * 4; i < items; i += THREADS * 4)
    *reinterpret_cast<float4*>(mine + i) = *reinterpret_cast<const float4*>(sums + i / STRIP * RP + i % STRIP);
  const long long q0 = static_cast<long long>(s) * C;
  const int c0 = split_cta(sp, q0), c1 = split_cta(sp, q0 + C - 1);
  int last = 0;
  if (THREADS == 32) __syncwarp();
  else bar_consumers<THREADS>();
  if (i0 == 0) {
    last = arrive_acq_rel(p.cnt + c0) == c1 - c0;
    if (last) p.cnt[c0] = 0;
    *flag = last;
  }
  if (THREADS == 32) {
    last = __shfl_sync(0xffffffffu, last, 0);
    __syncwarp();  // what lane 0 acquired
  } else {
    bar_consumers<THREADS>();
    last = *reinterpret_cast<volatile int*>(flag);
  }
  if (!last) return;
  // four columns a thread, several parts on their way at a time; the sums, in the place
  // of this CTA's own, are then written as above
  const int items4 = items / 4;
  const float4* head = reinterpret_cast<const float4*>(p.part) + (static_cast<size_t>(c0) * 2 + 1) * items4;
  const float4* rest = reinterpret_cast<const float4*>(p.part) + static_cast<size_t>(c0 + 1) * 2 * items4;
  // (one row of 2048 x 2048 in a graph: 5.8 us, with four and two as for the wide strips
  // 6.8; 13 rows of 2816 x 4224: 12.6, with one and eight 14.2: the code is run once and
  // waits for itself)
  constexpr int U = STRIP > kLinStrip ? 4 : 1, V = STRIP > kLinStrip ? 2 : 4;
#pragma unroll 1
  for (int i = i0; i < items4; i += U * THREADS) {
    float4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = i + j * THREADS < items4 ? __ldcg(head + i + j * THREADS) : float4{};
#pragma unroll 1
    for (int cta = 0; cta < c1 - c0; cta += V) {
      float4 w[V][U];
#pragma unroll
      for (int c = 0; c < V; ++c)
#pragma unroll
        for (int j = 0; j < U; ++j)
          w[c][j] = cta + c < c1 - c0 && i + j * THREADS < items4
                        ? __ldcg(rest + static_cast<size_t>(cta + c) * 2 * items4 + i + j * THREADS)
                        : float4{};
#pragma unroll
      for (int c = 0; c < V; ++c)
#pragma unroll
        for (int j = 0; j < U; ++j) {
          v[j].x += w[c][j].x;
          v[j].y += w[c][j].y;
          v[j].z += w[c][j].z;
          v[j].w += w[c][j].w;
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int o = (i + j * THREADS) * 4;
      if (o < items) *reinterpret_cast<float4*>(sums + o / STRIP * RP + o % STRIP) = v[j];
    }
  }
  if (THREADS == 32) __syncwarp();
  else bar_consumers<THREADS>();
  lin_write<THREADS, STRIP, TY>(p, sums, RP, s, i0);
}

cudaError_t launch_linear_w4_wide(int group, const CUtensorMap& mw, const LinParams& p, bool f32, cudaStream_t s);

}  // namespace moe
