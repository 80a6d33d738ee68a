// Low-rank adapters of many requests beside a shared projection (moe_lora):
//
//   y[t] = base[t] + scales[a] (x[t] A_a^T) B_a^T,   a = ids[t]
//
// Rows are taken in tiles of one adapter each.  Up to kLoraScanRows rows a CTA finds its
// tile in the ids by itself (the tile of row t is that of all rows with its adapter, and
// only the first of them has one); beyond, a launch sorts the rows by adapter and lists
// the tiles.  Then two launches: lora_shrink, v = x A^T as fp32 planes over slices of K, and
// lora_expand, which adds the planes in order and multiplies by B.
//
// Both products are mma.sync on operands that go from global memory straight to the
// registers that multiply them: A and B are row after row of the reduction dimension, as
// are x and v, and since a sum may take its terms in any order, a thread's four-byte pieces
// of a 32-wide step are taken from the 16 bytes that it loads.  At ranks of 8 to 256 the
// products are a small part of the time that x, y and the adapters' bytes need.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "moe_internal.h"
#include "stream_sm103.cuh"

namespace moe {
namespace {

constexpr int kLoraScanRows = 64;
constexpr int kLoraWarps = 8;
constexpr int kRankSlice = 64;  // columns of v that one warp holds sums of

struct LoraTile {
  int adapter;  // -1: rows without one
  int first;    // in the sorted rows
  int count;
};

struct LoraParams {
  const __nv_bfloat16 *x, *A, *B;
  const int32_t* ids;
  const float* scales;
  const void* base;
  void* y;
  float* planes;  // [splits, T, r]
  int32_t* order;
  LoraTile* tiles;
  int32_t* ntiles;
  int T, K, N, r, n;
  int splits;  // of K
  int slices;  // of r
  int chunk;   // columns of y a CTA takes, a multiple of 32 * kLoraWarps
};

// ------------------------------------------------------------------- plan
// One CTA: rows counted by adapter, adapters' starts, tiles of at most 16 MT rows, rows
// scattered (in any order inside an adapter: what a row gets does not depend on the rows
// beside it).
__global__ void __launch_bounds__(1024) lora_plan_kernel(const LoraParams p, int tile_rows) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ int32_t bins[];  // n + 1 counts, then next free positions
  __shared__ int2 warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nb = p.n + 1;
  for (int i = tid; i < nb; i += 1024) bins[i] = 0;
  __syncthreads();
  auto bin = [&](int id) { return static_cast<unsigned>(id) < static_cast<unsigned>(p.n) ? id : p.n; };
  // position of row t in its adapter's bin (t past the last: none).  A request's rows lie
  // together: one atomic for a warp whose rows have one adapter.
  auto take = [&](int t) {
    const bool in = t < p.T;
    const int b = in ? bin(p.ids[t]) : -1, b0 = __shfl_sync(0xffffffffu, b, 0);
    const unsigned mask = __ballot_sync(0xffffffffu, in);
    int at = 0;
    if (__all_sync(0xffffffffu, b == b0 || !in)) {
      if (lane == 0 && in) at = atomicAdd(&bins[b], __popc(mask));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << lane) - 1u));
    } else if (in) {
      at = atomicAdd(&bins[b], 1);
    }
    return at;
  };
  for (int t = tid; t - tid < p.T; t += 1024) take(t);
  __syncthreads();
  // exclusive sums of rows and of tiles over the adapters, a run of them a thread
  const int per = (nb + 1023) / 1024, b0 = min(nb, tid * per), b1 = min(nb, b0 + per);
  int rows = 0, tiles = 0;
  for (int b = b0; b < b1; ++b) {
    rows += bins[b];
    tiles += (bins[b] + tile_rows - 1) / tile_rows;
  }
  int2 inc = make_int2(rows, tiles);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, inc.x, o), c = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) {
      inc.x += a;
      inc.y += c;
    }
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int row = inc.x - rows, tile = inc.y - tiles;
  for (int w = 0; w < warp; ++w) {
    row += warp_sum[w].x;
    tile += warp_sum[w].y;
  }
  for (int b = b0; b < b1; ++b) {
    const int c = bins[b];
    for (int i = 0; i < c; i += tile_rows)
      p.tiles[tile++] = LoraTile{b < p.n ? b : -1, row + i, min(tile_rows, c - i)};
    bins[b] = row;
    row += c;
  }
  if (tid == 1023) *p.ntiles = tile;
  __syncthreads();
  for (int t = tid; t - tid < p.T; t += 1024) {
    const int at = take(t);
    if (t < p.T) p.order[at] = t;
  }
}

// --------------------------------------------------------------- tile rows
// The CTA's tile: its rows' numbers in `rows` (at most max_rows of them), its adapter;
// false when it has none.  Without a plan (SCAN) the tile is all rows with row b's adapter.
template <bool SCAN>
__device__ __forceinline__ bool lora_tile(const LoraParams& p, int b, int* rows, int* count_slot, int& adapter,
                                          int& count) {
  if (SCAN) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
      auto id = [&](int t) {
        const int a = t < p.T ? p.ids[t] : -2;
        return static_cast<unsigned>(a) < static_cast<unsigned>(p.n) ? a : t < p.T ? -1 : -2;
      };
      const int i0 = id(lane), i1 = id(lane + 32);
      const int mine = b < 32 ? __shfl_sync(0xffffffffu, i0, b) : __shfl_sync(0xffffffffu, i1, b - 32);
      const unsigned m0 = __ballot_sync(0xffffffffu, i0 == mine), m1 = __ballot_sync(0xffffffffu, i1 == mine);
      const int first = m0 ? __ffs(m0) - 1 : 32 + __ffs(m1) - 1;
      const unsigned below = (1u << lane) - 1u;
      if (i0 == mine) rows[__popc(m0 & below)] = lane;
      if (i1 == mine) rows[__popc(m0) + __popc(m1 & below)] = lane + 32;
      if (lane == 0) {
        count_slot[0] = first == b ? __popc(m0) + __popc(m1) : 0;
        count_slot[1] = mine;
      }
    }
    __syncthreads();
    count = count_slot[0];
    adapter = count_slot[1];
    return count > 0;
  }
  if (b >= *p.ntiles) return false;
  const LoraTile t = p.tiles[b];
  adapter = t.adapter;
  count = t.count;
  if (threadIdx.x < t.count) rows[threadIdx.x] = p.order[t.first + threadIdx.x];
  __syncthreads();
  return true;
}

__device__ __forceinline__ uint4 ldg16(const __nv_bfloat16* p, bool ok) {
  return ok ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}
// One 32-wide step of the reduction: D (16 x 8) += rows (g, g + 8) x column
__device__ __forceinline__ void step32(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& col) {
  mma_16816<false>(d, lo.x, hi.x, lo.y, hi.y, col.x, col.y);
  mma_16816<false>(d, lo.z, hi.z, lo.w, hi.w, col.z, col.w);
}

// ------------------------------------------------------------------ shrink
// planes[split][t][j] = sum over the split's k of x[t, k] A[a, j, k].  A CTA: a tile, a slice
// of at most 64 columns, a slice of K, whose 32-wide steps its warps take in turn; their sums
// are added in the order of the warps.
template <int MT, int NT, bool SCAN>
__global__ void __launch_bounds__(kLoraWarps * 32) lora_shrink_kernel(const LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int rows[SCAN ? kLoraScanRows : 16 * MT];
  __shared__ int slot[2];
  __shared__ float red[kLoraWarps][32][4 * NT + 1];
  int adapter, count;
  if (!lora_tile<SCAN>(p, blockIdx.x, rows, slot, adapter, count) || adapter < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int slice = blockIdx.y % p.slices, split = blockIdx.y / p.slices;
  const int j0 = slice * kRankSlice;
  const int steps = (p.K + 31) / 32, s0 = static_cast<long long>(steps) * split / p.splits,
            s1 = static_cast<long long>(steps) * (split + 1) / p.splits;
  const __nv_bfloat16* A = p.A + (static_cast<size_t>(adapter) * p.r + j0) * p.K;
  float* plane = p.planes + static_cast<size_t>(split) * p.T * p.r;
  for (int m0 = 0; m0 < count; m0 += 16 * MT) {
    const __nv_bfloat16* xr[MT][2];
    bool on[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m0 + 16 * m + 8 * h + g;
        on[m][h] = i < count;
        xr[m][h] = p.x + static_cast<size_t>(on[m][h] ? rows[i] : 0) * p.K;
      }
    float acc[MT][NT][4] = {};
    for (int s = s0 + warp; s < s1; s += kLoraWarps) {
      const int k = 32 * s + 8 * tig;
      const bool in = k < p.K;
      uint4 xa[MT][2], col[NT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) xa[m][h] = ldg16(xr[m][h] + k, in && on[m][h]);
#pragma unroll
      for (int j = 0; j < NT; ++j) col[j] = ldg16(A + static_cast<size_t>(8 * j + g) * p.K + k, in && j0 + 8 * j < p.r);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) step32(acc[m][j], xa[m][0], xa[m][1], col[j]);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][lane][4 * j + i] = acc[m][j][i];
      __syncthreads();
      for (int o = threadIdx.x; o < 16 * 8 * NT; o += kLoraWarps * 32) {
        const int i = o / (8 * NT), c = o % (8 * NT);  // row and column of the 16 x 8 NT tile
        const int l = 4 * (i & 7) + ((c & 7) >> 1), e = 4 * (c >> 3) + 2 * (i >> 3) + (c & 1);
        float v = red[0][l][e];
#pragma unroll
        for (int w = 1; w < kLoraWarps; ++w) v += red[w][l][e];
        const int at = m0 + 16 * m + i;
        if (at < count && j0 + c < p.r) plane[static_cast<size_t>(rows[at]) * p.r + j0 + c] = v;
      }
    }
  }
}

// ------------------------------------------------------------------ expand
// A CTA: a tile and `chunk` columns of y, whose 32-wide blocks its warps take in turn.  v is
// kept in shared memory as TERMS bf16 terms.  The eight columns of an instruction are spread
// so that a thread's four of them hold eight neighbouring columns of y.
template <int MT, int TERMS, bool SCAN, typename Ty>
__global__ void __launch_bounds__(kLoraWarps * 32) lora_expand_kernel(const LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int rows[SCAN ? kLoraScanRows : 16 * MT];
  __shared__ int slot[2];
  extern __shared__ __align__(16) __nv_bfloat16 vs[];  // [TERMS][16 MT][ld]
  int adapter, count;
  if (!lora_tile<SCAN>(p, blockIdx.x, rows, slot, adapter, count)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int c0 = blockIdx.y * p.chunk, c1 = min(p.N, c0 + p.chunk);
  const Ty* base = static_cast<const Ty*>(p.base);
  Ty* y = static_cast<Ty*>(p.y);
  if (adapter < 0) {
    if (base == y) return;
    constexpr int V = 16 / sizeof(Ty);
    const int nv = (c1 - c0) / V;
    for (int i = threadIdx.x; i < count * nv; i += kLoraWarps * 32) {
      const size_t at = static_cast<size_t>(rows[i / nv]) * p.N + c0 + V * (i % nv);
      *reinterpret_cast<uint4*>(y + at) = base ? *reinterpret_cast<const uint4*>(base + at) : make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int rp = (p.r + 31) / 32 * 32, ld = rp + 8;
  const float scale = p.scales ? p.scales[adapter] : 1.0f;
  const __nv_bfloat16* B = p.B + static_cast<size_t>(adapter) * p.N * p.r;
  for (int m0 = 0; m0 < count; m0 += 16 * MT) {
    if (m0) __syncthreads();
    for (int o = threadIdx.x; o < 16 * MT * rp; o += kLoraWarps * 32) {
      const int i = o / rp, j = o % rp;
      float v = 0.0f;
      if (m0 + i < count && j < p.r) {
        const float* q = p.planes + static_cast<size_t>(rows[m0 + i]) * p.r + j;
        for (int s = 0; s < p.splits; ++s) v += q[static_cast<size_t>(s) * p.T * p.r];
        v *= scale;
      }
#pragma unroll
      for (int z = 0; z < TERMS; ++z) {
        const __nv_bfloat16 b = __float2bfloat16_rn(v);
        vs[(z * 16 * MT + i) * ld + j] = b;
        const float f = __bfloat162float(b);
        v = isfinite(f) ? v - f : 0.0f;
      }
    }
    __syncthreads();
    for (int n0 = c0 + 32 * warp; n0 < c1; n0 += 32 * kLoraWarps) {
      float acc[MT][4][4] = {};
      for (int r0 = 0; r0 < rp; r0 += 32) {
        const int k = r0 + 8 * tig;
        uint4 col[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
          col[j] = ldg16(B + static_cast<size_t>(n) * p.r + k, n < p.N && k < p.r);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int z = 0; z < TERMS; ++z) {
            const __nv_bfloat16* a = vs + (z * 16 * MT + 16 * m + g) * ld + k;
            const uint4 lo = *reinterpret_cast<const uint4*>(a), hi = *reinterpret_cast<const uint4*>(a + 8 * ld);
#pragma unroll
            for (int j = 0; j < 4; ++j) step32(acc[m][j], lo, hi, col[j]);
          }
      }
      const int n = n0 + 8 * tig;
      if (n >= c1) continue;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = m0 + 16 * m + 8 * h + g;
          if (i >= count) continue;
          const size_t at = static_cast<size_t>(rows[i]) * p.N + n;
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[2 * j] = acc[m][j][2 * h];
            f[2 * j + 1] = acc[m][j][2 * h + 1];
          }
          if constexpr (sizeof(Ty) == 2) {
            if (base) {
              const uint4 w = *reinterpret_cast<const uint4*>(base + at);
              const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                f[2 * j] += __uint_as_float(u[j] << 16);
                f[2 * j + 1] += __uint_as_float(u[j] & 0xffff0000u);
              }
            }
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
              u[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(y + at) = make_uint4(u[0], u[1], u[2], u[3]);
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float4 w = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
              if (base) {
                const float4 b = *reinterpret_cast<const float4*>(base + at + 4 * q);
                w.x += b.x;
                w.y += b.y;
                w.z += b.z;
                w.w += b.w;
              }
              *reinterpret_cast<float4*>(y + at + 4 * q) = w;
            }
          }
        }
    }
  }
}

constexpr int kSms = 152;  // a constant: results must not depend on the device

int tile_mt(int T, int n) { return T > kLoraScanRows && T >= 16 * n ? 2 : 1; }
// most tiles that T rows can have
int max_tiles(int T, int n) {
  if (T <= kLoraScanRows) return T;
  const int rows = 16 * tile_mt(T, n);
  return static_cast<int>(std::min<long long>(T, (T + rows - 1ll) / rows + n));
}

struct LoraLayout {
  size_t planes, order, tiles, ntiles, total;
  int splits, slices, chunk;
};
LoraLayout lora_layout(int T, int K, int N, int r, int n) {
  LoraLayout L{};
  const long long tiles = std::max(1, T <= kLoraScanRows ? std::min(T, n) : max_tiles(T, n));
  L.slices = (r + kRankSlice - 1) / kRankSlice;
  // two CTAs an SM, a step at least for each warp of a split
  const int steps = (K + 31) / 32;
  L.splits = static_cast<int>(std::max(1ll, std::min<long long>(2 * kSms / (tiles * L.slices), steps / kLoraWarps)));
  // four CTAs an SM, a block of 32 columns at least for each warp
  const int unit = 32 * kLoraWarps, units = (N + unit - 1) / unit;
  const int chunks = static_cast<int>(std::max(1ll, std::min<long long>(4 * kSms / tiles, units)));
  L.chunk = (units + chunks - 1) / chunks * unit;
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur = (cur + bytes + 255) / 256 * 256;
    return o;
  };
  L.planes = take(static_cast<size_t>(L.splits) * T * r * 4);
  L.order = take(static_cast<size_t>(T) * 4);
  L.tiles = take(static_cast<size_t>(max_tiles(T, n)) * sizeof(LoraTile));
  L.ntiles = take(4);
  L.total = cur;
  return L;
}

template <int MT, int NT, bool SCAN>
cudaError_t shrink(const LoraParams& p, dim3 grid, cudaStream_t s) {
  return launch_kernel(lora_shrink_kernel<MT, NT, SCAN>, grid, dim3(kLoraWarps * 32), 0, s, p);
}
template <int MT, bool SCAN>
cudaError_t shrink_rank(const LoraParams& p, dim3 grid, cudaStream_t s) {
  if (p.r <= 16) return shrink<MT, 2, SCAN>(p, grid, s);
  if (p.r <= 32) return shrink<MT, 4, SCAN>(p, grid, s);
  return shrink<MT, 8, SCAN>(p, grid, s);
}
template <int MT, int TERMS, bool SCAN, typename Ty>
cudaError_t expand(const LoraParams& p, dim3 grid, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(TERMS) * 16 * MT * ((p.r + 31) / 32 * 32 + 8) * 2;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(lora_expand_kernel<MT, TERMS, SCAN, Ty>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(lora_expand_kernel<MT, TERMS, SCAN, Ty>, grid, dim3(kLoraWarps * 32), smem, s, p);
}
template <int MT, bool SCAN>
cudaError_t products(const LoraParams& p, int tiles, bool y_f32, cudaStream_t s) {
  cudaError_t e = shrink_rank<MT, SCAN>(p, dim3(tiles, p.splits * p.slices), s);
  if (e != cudaSuccess) return e;
  const dim3 grid(tiles, (p.N + p.chunk - 1) / p.chunk);
  e = y_f32 ? expand<MT, 3, SCAN, float>(p, grid, s) : expand<MT, 2, SCAN, __nv_bfloat16>(p, grid, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int T, int K, int N, int r, int n) { return std::max<size_t>(256, lora_layout(T, K, N, r, n).total); }

cudaError_t launch_lora(int T, int K, int N, int r, int n, const void* x, const int32_t* ids, const void* A,
                        const void* B, const float* scales, const void* base, void* y, bool y_f32, uint8_t* ws,
                        cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  const LoraLayout L = lora_layout(T, K, N, r, n);
  LoraParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.A = static_cast<const __nv_bfloat16*>(A);
  p.B = static_cast<const __nv_bfloat16*>(B);
  p.ids = ids;
  p.scales = scales;
  p.base = base;
  p.y = y;
  p.planes = reinterpret_cast<float*>(ws + L.planes);
  p.order = reinterpret_cast<int32_t*>(ws + L.order);
  p.tiles = reinterpret_cast<LoraTile*>(ws + L.tiles);
  p.ntiles = reinterpret_cast<int32_t*>(ws + L.ntiles);
  p.T = T;
  p.K = K;
  p.N = N;
  p.r = r;
  p.n = n;
  p.splits = L.splits;
  p.slices = L.slices;
  p.chunk = L.chunk;
  const int tiles = max_tiles(T, n);
  if (T <= kLoraScanRows) return products<1, true>(p, tiles, y_f32, s);
  const int mt = tile_mt(T, n);
  const size_t smem = static_cast<size_t>(n + 1) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(lora_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((kLoraMaxAdapters + 1) * 4));
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_kernel(lora_plan_kernel, dim3(1), dim3(1024), smem, s, p, 16 * mt);
  if (e != cudaSuccess) return e;
  return mt == 2 ? products<2, false>(p, tiles, y_f32, s) : products<1, false>(p, tiles, y_f32, s);
}

}  // namespace moe
