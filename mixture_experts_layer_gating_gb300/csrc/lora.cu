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
#include "sm103_ptx.cuh"
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
  int chunk;   // columns of y a CTA takes, a multiple of 256
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
  if (static_cast<int>(threadIdx.x) < t.count) rows[threadIdx.x] = p.order[t.first + threadIdx.x];
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

// ---------------------------------------------------- shrink, a few rows to a tile
// planes[split][t][j] = sum over the split's k of x[t, k] A[a, j, k].  A CTA: a tile, a slice
// of at most 64 columns, a slice of K, whose 32-wide steps its warps take in turn, two at a
// time so that both steps' loads are under way; their sums are added in the order of the
// warps.
template <int NT, bool SCAN>
__global__ void __launch_bounds__(kLoraWarps * 32, 2) lora_shrink_kernel(const LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int rows[SCAN ? kLoraScanRows : 16];
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
  for (int m0 = 0; m0 < count; m0 += 16) {
    const bool on0 = m0 + g < count, on1 = m0 + 8 + g < count;
    const __nv_bfloat16* x0 = p.x + static_cast<size_t>(on0 ? rows[m0 + g] : 0) * p.K;
    const __nv_bfloat16* x1 = p.x + static_cast<size_t>(on1 ? rows[m0 + 8 + g] : 0) * p.K;
    float acc[NT][4] = {};
    for (int s = s0 + warp; s < s1; s += 2 * kLoraWarps) {
      uint4 lo[2], hi[2], col[2][NT];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = 32 * (s + u * kLoraWarps) + 8 * tig;
        const bool in = k < p.K && (u == 0 || s + kLoraWarps < s1);
        lo[u] = ldg16(x0 + k, in && on0);
        hi[u] = ldg16(x1 + k, in && on1);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          col[u][j] = ldg16(A + static_cast<size_t>(8 * j + g) * p.K + k, in && j0 + 8 * j < p.r);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < NT; ++j) step32(acc[j], lo[u], hi[u], col[u][j]);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][lane][4 * j + i] = acc[j][i];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * 8 * NT; o += kLoraWarps * 32) {
      const int i = o / (8 * NT), c = o % (8 * NT);  // row and column of the 16 x 8 NT tile
      const int l = 4 * (i & 7) + ((c & 7) >> 1), e = 4 * (c >> 3) + 2 * (i >> 3) + (c & 1);
      float v = red[0][l][e];
#pragma unroll
      for (int w = 1; w < kLoraWarps; ++w) v += red[w][l][e];
      if (m0 + i < count && j0 + c < p.r) plane[static_cast<size_t>(rows[m0 + i]) * p.r + j0 + c] = v;
    }
  }
}

// y = base + f for 8 neighbouring values; b: the base's, as loaded (not read where !has).
__device__ __forceinline__ void put8(__nv_bfloat16* y, float (&f)[8], bool has, const uint4 (&b)[1]) {
  if (has) {
    const uint32_t u[4] = {b[0].x, b[0].y, b[0].z, b[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] += __uint_as_float(u[j] << 16);
      f[2 * j + 1] += __uint_as_float(u[j] & 0xffff0000u);
    }
  }
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    u[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(y) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void put8(float* y, float (&f)[8], bool has, const uint4 (&b)[2]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float4 w = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
    if (has) {
      w.x += __uint_as_float(b[q].x);
      w.y += __uint_as_float(b[q].y);
      w.z += __uint_as_float(b[q].z);
      w.w += __uint_as_float(b[q].w);
    }
    reinterpret_cast<float4*>(y)[q] = w;
  }
}

// Rows without an adapter: columns [c0, c1) of their base, copied (nothing where y is the base).
template <typename Ty>
__device__ __forceinline__ void copy_rows(const Ty* base, Ty* y, const int* rows, int count, int N, int c0, int c1) {
  if (base == y) return;
  constexpr int V = 16 / sizeof(Ty);
  const int nv = (c1 - c0) / V;
  for (int i = threadIdx.x; i < count * nv; i += blockDim.x) {
    const size_t at = static_cast<size_t>(rows[i / nv]) * N + c0 + V * (i % nv);
    *reinterpret_cast<uint4*>(y + at) = base ? *reinterpret_cast<const uint4*>(base + at) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// f[0..7] = v[row][j .. j + 7]: the planes added in their order, four planes' loads at a time.
__device__ __forceinline__ void sum_planes(const LoraParams& p, int row, int j, float (&f)[8]) {
  const float* q = p.planes + static_cast<size_t>(row) * p.r + j;
  const size_t plane = static_cast<size_t>(p.T) * p.r;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  for (int s = 0; s < p.splits; s += 4) {
    float4 a[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s + u < p.splits) {
        a[u][0] = *reinterpret_cast<const float4*>(q + (s + u) * plane);
        a[u][1] = *reinterpret_cast<const float4*>(q + (s + u) * plane + 4);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s + u < p.splits)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f[4 * h] += a[u][h].x;
          f[4 * h + 1] += a[u][h].y;
          f[4 * h + 2] += a[u][h].z;
          f[4 * h + 3] += a[u][h].w;
        }
  }
}
// f as TERMS bf16 terms, 8 values to a word of 16 bytes; f keeps what is left.
template <int TERMS>
__device__ __forceinline__ void split_terms(float (&f)[8], uint4 (&t)[TERMS]) {
#pragma unroll
  for (int z = 0; z < TERMS; ++z) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 b = __bfloat1622float2(h);
      // (past bf16's range the first term is infinite and the others are 0)
      f[2 * j] = isfinite(b.x) ? f[2 * j] - b.x : 0.0f;
      f[2 * j + 1] = isfinite(b.y) ? f[2 * j + 1] - b.y : 0.0f;
    }
    t[z] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// ---------------------------------------------------- expand, a few rows to a tile
// A CTA: a tile and `chunk` columns of y, whose 32-wide blocks its warps take in turn.  v is
// kept in shared memory as TERMS bf16 terms.  The eight columns of an instruction are spread
// so that a thread's four of them hold eight neighbouring columns of y.  The first block's
// part of B is loaded before the planes are waited for: of what this launch reads only they
// come from the one before it, which itself began after all that went before.
template <int TERMS, bool SCAN, typename Ty>
__global__ void __launch_bounds__(kLoraWarps * 32, 2) lora_expand_kernel(const LoraParams p) {
  __shared__ int rows[SCAN ? kLoraScanRows : 16];
  __shared__ int slot[2];
  extern __shared__ __align__(16) __nv_bfloat16 vs[];  // [TERMS][16][ld]
  int adapter, count;
  const bool tile = lora_tile<SCAN>(p, blockIdx.x, rows, slot, adapter, count);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int c0 = blockIdx.y * p.chunk, c1 = min(p.N, c0 + p.chunk);
  const Ty* base = static_cast<const Ty*>(p.base);
  Ty* y = static_cast<Ty*>(p.y);
  const int rp = (p.r + 31) / 32 * 32, ld = rp + 8;
  const __nv_bfloat16* B = p.B + static_cast<size_t>(tile && adapter > 0 ? adapter : 0) * p.N * p.r;
  // column of y that this thread's part of instruction j's B operand belongs to
  const int nb = 8 * (g >> 1) + (g & 1);
  auto load_cols = [&](uint4 (&col)[4], int n0, int r0) {
    const int k = r0 + 8 * tig;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + nb + 2 * j;
      col[j] = ldg16(B + static_cast<size_t>(n) * p.r + k, n < p.N && k < p.r);
    }
  };
  uint4 col[2][4];  // of 64 of the rank
  auto load_step = [&](int n0, int r0) {
    load_cols(col[0], n0, r0);
    load_cols(col[1], n0, r0 + 32);
  };
  const bool work = tile && adapter >= 0;
  const int n_first = c0 + 32 * warp;
  if (work) load_step(n_first, 0);
  pdl_wait();
  pdl_launch_dependents();
  if (!tile) return;
  if (!work) {
    copy_rows(base, y, rows, count, p.N, c0, c1);
    return;
  }
  const float scale = p.scales ? p.scales[adapter] : 1.0f;
  constexpr int W = sizeof(Ty) / 2;  // 16-byte words of eight values
  for (int m0 = 0; m0 < count; m0 += 16) {
    if (m0) {
      __syncthreads();
      load_step(n_first, 0);
    }
    for (int o = threadIdx.x; o < 2 * rp; o += kLoraWarps * 32) {
      const int i = o / (rp / 8), j = o % (rp / 8) * 8;
      float f[8] = {};
      if (m0 + i < count && j < p.r) {
        sum_planes(p, rows[m0 + i], j, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] *= scale;
      }
      uint4 t[TERMS];
      split_terms<TERMS>(f, t);
#pragma unroll
      for (int z = 0; z < TERMS; ++z) *reinterpret_cast<uint4*>(vs + (z * 16 + i) * ld + j) = t[z];
    }
    __syncthreads();
    for (int n0 = n_first; n0 < c1; n0 += 32 * kLoraWarps) {
      const int n = n0 + 8 * tig;
      uint4 b[2][W];
      size_t at[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m0 + 8 * h + g;
        at[h] = static_cast<size_t>(i < count ? rows[i] : 0) * p.N + n;
        if (base && i < count && n < c1) {
#pragma unroll
          for (int q = 0; q < W; ++q) b[h][q] = reinterpret_cast<const uint4*>(base + at[h])[q];
        }
      }
      float acc[4][4] = {};
      for (int r0 = 0; r0 < rp; r0 += 64) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (r0 + 32 * u >= rp) break;
#pragma unroll
          for (int z = 0; z < TERMS; ++z) {
            const __nv_bfloat16* a = vs + (z * 16 + g) * ld + r0 + 32 * u + 8 * tig;
            const uint4 lo = *reinterpret_cast<const uint4*>(a), hi = *reinterpret_cast<const uint4*>(a + 8 * ld);
#pragma unroll
            for (int j = 0; j < 4; ++j) step32(acc[j], lo, hi, col[u][j]);
          }
        }
        // the next step's, under way while this block is finished
        if (r0 + 64 < rp)
          load_step(n0, r0 + 64);
        else if (n0 + 32 * kLoraWarps < c1)
          load_step(n0 + 32 * kLoraWarps, 0);
      }
      if (n >= c1) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (m0 + 8 * h + g >= count) continue;
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = acc[j][2 * h];
          f[2 * j + 1] = acc[j][2 * h + 1];
        }
        put8(y + at[h], f, base != nullptr, b[h]);
      }
    }
  }
}

// --------------------------------------------------------- many rows to a tile
// Rings of shared-memory stages filled by cp.async, each stage's rows cut into 16-byte
// pieces.  Two neighbouring rows are read by a quarter of a warp at the same piece of
// each, so where they would meet in the banks odd rows keep their pieces in another order.
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// Shrink.  A CTA: a tile of at most BM rows, a slice of 8 NT RW columns of v and a slice of
// K.  Its four warps hold 32 rows x 8 NT columns each (RW of them beside one another).
constexpr int kShrinkStages = 4, kShrinkThreads = 128;
template <int BM, int NT>
struct ShrinkTile {
  static constexpr int RW = 4 * 32 / BM, COLS = 8 * NT * RW;
  static constexpr int kStage = (BM + COLS) * 128;  // 64 of K a stage
  static constexpr int kSmem = kShrinkStages * kStage;
};
template <int BM, int NT>
__global__ void __launch_bounds__(kShrinkThreads, 2) lora_shrink_wide_kernel(const LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  using Tile = ShrinkTile<BM, NT>;
  __shared__ int rows[BM];
  extern __shared__ __align__(128) uint8_t ring[];
  if (blockIdx.x >= *p.ntiles) return;
  const LoraTile tile = p.tiles[blockIdx.x];
  if (tile.adapter < 0) return;
  for (int i = threadIdx.x; i < BM; i += kShrinkThreads) rows[i] = i < tile.count ? p.order[tile.first + i] : -1;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int slice = blockIdx.y % p.slices, split = blockIdx.y / p.slices;
  const int j0 = slice * Tile::COLS;
  const int steps = (p.K + 63) / 64, s0 = static_cast<long long>(steps) * split / p.splits,
            s1 = static_cast<long long>(steps) * (split + 1) / p.splits;
  // this thread's piece of 16 bytes, of rows t0, t0 + 16, ...
  const int piece = threadIdx.x & 7, t0 = threadIdx.x >> 3;
  const uint32_t base = smem_u32(ring), put = t0 * 128 + ((piece ^ (4 * (t0 & 1))) << 4);
  const __nv_bfloat16* A = p.A + (static_cast<size_t>(tile.adapter) * p.r + j0) * p.K;
  int xrow[BM / 16];
#pragma unroll
  for (int i = 0; i < BM / 16; ++i) xrow[i] = rows[t0 + 16 * i];
  auto load = [&](int s) {
    if (s < s1) {
      const uint32_t to = base + static_cast<uint32_t>((s - s0) % kShrinkStages) * Tile::kStage + put;
      const int k = 64 * s + 8 * piece;
      const bool in = k < p.K;
#pragma unroll
      for (int i = 0; i < BM / 16; ++i) {
        const bool on = in && xrow[i] >= 0;
        cp_async_16(to + i * 2048, on ? p.x + static_cast<size_t>(xrow[i]) * p.K + k : p.x, on ? 16u : 0u);
      }
#pragma unroll
      for (int i = 0; i < (Tile::COLS + 15) / 16; ++i) {
        const int j = t0 + 16 * i;
        const bool on = in && j0 + j < p.r;
        cp_async_16(to + BM * 128 + i * 2048, on ? A + static_cast<size_t>(j) * p.K + k : p.x, on ? 16u : 0u);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kShrinkStages - 1; ++i) load(s0 + i);
  const int m0 = warp / Tile::RW * 32, c0 = warp % Tile::RW * 8 * NT;
  const uint32_t xat = base + (m0 + g) * 128, aat = base + (BM + c0 + g) * 128;
  float acc[2][NT][4] = {};
  for (int s = s0; s < s1; ++s) {
    cp_wait<kShrinkStages - 2>();
    __syncthreads();  // the stage is there, and every warp is done with the one filled next
    load(s + kShrinkStages - 1);
    const uint32_t stage = static_cast<uint32_t>((s - s0) % kShrinkStages) * Tile::kStage;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = stage + (((4 * h + tig) ^ (4 * (g & 1))) << 4);
      uint4 xa[2][2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        xa[m][0] = lds16(xat + at + m * 2048);
        xa[m][1] = lds16(xat + at + m * 2048 + 1024);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 col = lds16(aat + at + j * 1024);
#pragma unroll
        for (int m = 0; m < 2; ++m) step32(acc[m][j], xa[m][0], xa[m][1], col);
      }
    }
  }
  float* plane = p.planes + static_cast<size_t>(split) * p.T * p.r;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = rows[m0 + 16 * m + 8 * h + g];
      if (row < 0) continue;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (j0 + c0 + 8 * j < p.r)
          *reinterpret_cast<float2*>(plane + static_cast<size_t>(row) * p.r + j0 + c0 + 8 * j + 2 * tig) =
              make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
    }
}

// Expand.  A CTA: a tile and `chunk` columns of y in blocks of 128 bytes of a row of y (ranks
// past 64: 64 columns), whose rows of B and whose base come through the ring.  Eight warps of
// 16 rows each, or, for ranks past 64, two beside one another on each 16 rows.  v's terms stay in
// registers up to rank 64, past it in shared memory.
constexpr int kExpandThreads = 256;
template <typename Ty, bool HIGH>
struct ExpandTile {
  static constexpr int TERMS = sizeof(Ty) == 2 ? 2 : 3;
  static constexpr int BM = HIGH ? 64 : 128;
  static constexpr int COLS = HIGH ? 64 : 128 / sizeof(Ty);
  static constexpr int kStages = !HIGH ? 4 : sizeof(Ty) == 2 ? 3 : 2;  // (rank 256: 184 KB and 192 KB)
  static constexpr int kRow = COLS * sizeof(Ty);  // bytes of a row of the base
  static size_t smem(int rp) {
    return static_cast<size_t>(kStages) * (COLS * rp * 2 + BM * kRow) + (HIGH ? TERMS * BM * rp * 2 : 0);
  }
};
template <typename Ty, bool HIGH>
__global__ void __launch_bounds__(kExpandThreads, HIGH ? 1 : 2) lora_expand_wide_kernel(const LoraParams p) {
  using Tile = ExpandTile<Ty, HIGH>;
  constexpr int TERMS = Tile::TERMS, BM = Tile::BM, COLS = Tile::COLS, STAGES = Tile::kStages;
  constexpr int W = sizeof(Ty) / 2;  // 16-byte words of eight values
  __shared__ int rows[BM];
  extern __shared__ __align__(128) uint8_t ring[];
  const bool there = blockIdx.x < *p.ntiles;
  const LoraTile tile = there ? p.tiles[blockIdx.x] : LoraTile{-1, 0, 0};
  for (int i = threadIdx.x; i < BM; i += kExpandThreads) rows[i] = i < tile.count ? p.order[tile.first + i] : -1;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int c0 = blockIdx.y * p.chunk, c1 = min(p.N, c0 + p.chunk);
  const Ty* base = static_cast<const Ty*>(p.base);
  Ty* y = static_cast<Ty*>(p.y);
  const int rp = (p.r + 31) / 32 * 32, pieces = rp / 8;
  const int swz = rp & 32 ? 0 : 4;  // rows of an odd number of 64 bytes do not meet in the banks
  const uint32_t stage_bytes = COLS * rp * 2 + BM * Tile::kRow, smem = smem_u32(ring);
  const uint32_t terms_at = smem + STAGES * stage_bytes;
  const __nv_bfloat16* B = p.B + static_cast<size_t>(max(tile.adapter, 0)) * p.N * p.r;
  const int blocks = (c1 - c0 + COLS - 1) / COLS;
  auto load = [&](int b) {
    if (b < blocks) {
      const uint32_t to = smem + static_cast<uint32_t>(b % STAGES) * stage_bytes;
      const int n0 = c0 + b * COLS;
      for (int i = threadIdx.x; i < COLS * pieces; i += kExpandThreads) {
        const int n = i / pieces, c = i % pieces;
        const bool on = n0 + n < p.N && 8 * c < p.r;
        cp_async_16(to + n * rp * 2 + ((c ^ (swz * (n & 1))) << 4), on ? B + static_cast<size_t>(n0 + n) * p.r + 8 * c : p.B,
                    on ? 16u : 0u);
      }
      if (base) {
        constexpr int PR = Tile::kRow / 16;
#pragma unroll
        for (int u = 0; u < BM * PR / kExpandThreads; ++u) {
          const int i = threadIdx.x + u * kExpandThreads, t = i / PR, c = i % PR, n = n0 + c * 16 / static_cast<int>(sizeof(Ty));
          const int row = rows[t];
          const bool on = row >= 0 && n < p.N;
          cp_async_16(to + COLS * rp * 2 + t * Tile::kRow + ((c ^ ((W == 1 ? 4 : 1) * (t & 1))) << 4),
                      on ? base + static_cast<size_t>(row) * p.N + n : base, on ? 16u : 0u);
        }
      }
    }
    cp_commit();
  };
  if (there && tile.adapter >= 0) {  // nothing of these comes from the launch before (the planes do)
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) load(i);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (!there) return;
  if (tile.adapter < 0) {
    copy_rows(base, y, rows, tile.count, p.N, c0, c1);
    return;
  }
  const float scale = p.scales ? p.scales[tile.adapter] : 1.0f;
  const int mw = warp % (BM / 16), nw = warp / (BM / 16);
  const int row[2] = {rows[16 * mw + g], rows[16 * mw + 8 + g]};
  uint4 va[HIGH ? 1 : 2][2][TERMS];  // [32 of the rank][row half]
  if constexpr (HIGH) {
    for (int i = threadIdx.x; i < BM * pieces; i += kExpandThreads) {
      const int t = i / pieces, c = i % pieces;
      float f[8] = {};
      if (rows[t] >= 0 && 8 * c < p.r) {
        sum_planes(p, rows[t], 8 * c, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] *= scale;
      }
      uint4 term[TERMS];
      split_terms<TERMS>(f, term);
#pragma unroll
      for (int z = 0; z < TERMS; ++z)
        *reinterpret_cast<uint4*>(ring + STAGES * stage_bytes + ((z * BM + t) * pieces + (c ^ (swz * (t & 1)))) * 16) = term[z];
    }
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8] = {};
        if (row[h] >= 0 && 32 * u + 8 * tig < p.r) {
          sum_planes(p, row[h], 32 * u + 8 * tig, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) f[q] *= scale;
        }
        split_terms<TERMS>(f, va[u][h]);
      }
  }
  const int nb = 8 * (g >> 1) + (g & 1);
  constexpr int NBLK = HIGH ? 1 : COLS / 32;  // 32-wide blocks a warp takes of a stage
  for (int b = 0; b < blocks; ++b) {
    cp_wait<STAGES - 2>();
    __syncthreads();  // the stage (and v's terms) are there, and every warp is done with the one filled next
    load(b + STAGES - 1);
    const uint32_t stage = smem + static_cast<uint32_t>(b % STAGES) * stage_bytes;
#pragma unroll
    for (int q = 0; q < NBLK; ++q) {
      const int w0 = 32 * (HIGH ? nw : q);  // first column of the warp's block in the stage
      const uint32_t bat = stage + (w0 + nb) * rp * 2;
      float acc[4][4] = {};
      auto multiply = [&](int r0, const uint4 (&lo)[TERMS], const uint4 (&hi)[TERMS]) {
        const uint32_t c = ((r0 / 8 + tig) ^ (swz * (g & 1))) << 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 col = lds16(bat + 2 * j * rp * 2 + c);
#pragma unroll
          for (int z = 0; z < TERMS; ++z) step32(acc[j], lo[z], hi[z], col);
        }
      };
      if constexpr (HIGH) {
        for (int r0 = 0; r0 < rp; r0 += 32) {
          uint4 lo[TERMS], hi[TERMS];
          const uint32_t c = ((r0 / 8 + tig) ^ (swz * (g & 1))) << 4;
#pragma unroll
          for (int z = 0; z < TERMS; ++z) {
            lo[z] = lds16(terms_at + (z * BM + 16 * mw + g) * rp * 2 + c);
            hi[z] = lds16(terms_at + (z * BM + 16 * mw + 8 + g) * rp * 2 + c);
          }
          multiply(r0, lo, hi);
        }
      } else {
        multiply(0, va[0][0], va[0][1]);
        if (rp > 32) multiply(32, va[1][0], va[1][1]);
      }
      const int n = c0 + b * COLS + w0 + 8 * tig;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (row[h] < 0 || n >= c1) continue;
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = acc[j][2 * h];
          f[2 * j + 1] = acc[j][2 * h + 1];
        }
        uint4 w[W];
        if (base) {
          const int t = 16 * mw + 8 * h + g;
#pragma unroll
          for (int i = 0; i < W; ++i)
            w[i] = lds16(stage + COLS * rp * 2 + t * Tile::kRow +
                         (((W * (w0 / 8 + tig) + i) ^ ((W == 1 ? 4 : 1) * (t & 1))) << 4));
        }
        put8(y + static_cast<size_t>(row[h]) * p.N + n, f, base != nullptr, w);
      }
    }
  }
}

constexpr int kSms = 152;  // a constant: results must not depend on the device

// How T rows of n adapters are taken: `scan`, tiles found by the CTAs themselves; `wide`, the
// kernels for many rows to a tile (at least 32 rows an adapter on average).
struct LoraPlan {
  bool scan, wide;
  int tile_rows, tiles, slice_cols, slices, splits, chunk;
};
LoraPlan lora_plan(int T, int K, int N, int r, int n) {
  LoraPlan q{};
  q.scan = T <= kLoraScanRows;
  q.wide = !q.scan && T >= 32ll * n;
  q.tile_rows = !q.wide ? 16 : r <= 64 ? 128 : 64;
  q.tiles = q.scan ? T : static_cast<int>(std::min<long long>(T, (T + q.tile_rows - 1ll) / q.tile_rows + n));
  // tiles with an adapter, about
  const long long tiles = std::max(1, q.scan ? std::min(T, n) : q.wide ? (T + q.tile_rows - 1) / q.tile_rows + n / 2 : q.tiles);
  q.slice_cols = q.wide ? (r <= 16 ? 16 : r <= 32 ? 32 : 64) : kRankSlice;
  q.slices = (r + q.slice_cols - 1) / q.slice_cols;
  // two CTAs an SM; a step at least for each warp of a split, or four stages
  const int most = q.wide ? (K + 255) / 256 : (K + 32 * kLoraWarps - 1) / (32 * kLoraWarps);
  q.splits = static_cast<int>(std::max(1ll, std::min<long long>(2 * kSms / (tiles * q.slices), most)));
  // wide: two CTAs an SM, of four blocks at least; else four CTAs an SM, a block of 32 columns at
  // least for each warp
  const int unit = q.wide ? 256 : 32 * kLoraWarps, units = (N + unit - 1) / unit;
  const int chunks = static_cast<int>(std::max(1ll, std::min<long long>((q.wide ? 2 : 4) * kSms / tiles, units)));
  q.chunk = (units + chunks - 1) / chunks * unit;
  return q;
}

struct LoraLayout {
  size_t planes, order, tiles, ntiles, total;
};
LoraLayout lora_layout(const LoraPlan& q, int T, int r) {
  LoraLayout L{};
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur = (cur + bytes + 255) / 256 * 256;
    return o;
  };
  L.planes = take(static_cast<size_t>(q.splits) * T * r * 4);
  if (!q.scan) {
    L.order = take(static_cast<size_t>(T) * 4);
    L.tiles = take(static_cast<size_t>(q.tiles) * sizeof(LoraTile));
    L.ntiles = take(4);
  }
  L.total = std::max<size_t>(cur, 256);
  return L;
}

// More shared memory than a launch gets unasked.
template <typename Kernel>
cudaError_t allow_smem(Kernel* kern, size_t bytes) {
  return bytes <= 48 * 1024 ? cudaSuccess
                            : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <bool SCAN>
cudaError_t products(const LoraParams& p, const LoraPlan& q, bool y_f32, cudaStream_t s) {
  const dim3 block(kLoraWarps * 32), grid(q.tiles, p.splits * p.slices), egrid(q.tiles, (p.N + p.chunk - 1) / p.chunk);
  auto shrink = p.r <= 16 ? lora_shrink_kernel<2, SCAN> : p.r <= 32 ? lora_shrink_kernel<4, SCAN> : lora_shrink_kernel<8, SCAN>;
  cudaError_t e = launch_kernel(shrink, grid, block, 0, s, p);
  if (e != cudaSuccess) return e;
  auto expand = y_f32 ? lora_expand_kernel<3, SCAN, float> : lora_expand_kernel<2, SCAN, __nv_bfloat16>;
  const size_t smem = static_cast<size_t>(y_f32 ? 3 : 2) * 16 * ((p.r + 31) / 32 * 32 + 8) * 2;
  e = launch_kernel(expand, egrid, block, smem, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int BM, int NT>
cudaError_t shrink_wide(const LoraParams& p, const LoraPlan& q, cudaStream_t s) {
  constexpr size_t smem = ShrinkTile<BM, NT>::kSmem;
  const cudaError_t e = allow_smem(lora_shrink_wide_kernel<BM, NT>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(lora_shrink_wide_kernel<BM, NT>, dim3(q.tiles, p.splits * p.slices), dim3(kShrinkThreads), smem, s, p);
}
template <typename Ty, bool HIGH>
cudaError_t expand_wide(const LoraParams& p, const LoraPlan& q, cudaStream_t s) {
  const size_t smem = ExpandTile<Ty, HIGH>::smem((p.r + 31) / 32 * 32);
  const cudaError_t e = allow_smem(lora_expand_wide_kernel<Ty, HIGH>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(lora_expand_wide_kernel<Ty, HIGH>, dim3(q.tiles, (p.N + p.chunk - 1) / p.chunk), dim3(kExpandThreads),
                       smem, s, p);
}
cudaError_t products_wide(const LoraParams& p, const LoraPlan& q, bool y_f32, cudaStream_t s) {
  cudaError_t e = p.r > 64    ? shrink_wide<64, 4>(p, q, s)
                  : p.r > 32  ? shrink_wide<128, 8>(p, q, s)
                  : p.r > 16  ? shrink_wide<128, 4>(p, q, s)
                              : shrink_wide<128, 2>(p, q, s);
  if (e != cudaSuccess) return e;
  if (p.r > 64)
    e = y_f32 ? expand_wide<float, true>(p, q, s) : expand_wide<__nv_bfloat16, true>(p, q, s);
  else
    e = y_f32 ? expand_wide<float, false>(p, q, s) : expand_wide<__nv_bfloat16, false>(p, q, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int T, int K, int N, int r, int n) { return lora_layout(lora_plan(T, K, N, r, n), T, r).total; }

cudaError_t launch_lora(int T, int K, int N, int r, int n, const void* x, const int32_t* ids, const void* A,
                        const void* B, const float* scales, const void* base, void* y, bool y_f32, uint8_t* ws,
                        cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  const LoraPlan q = lora_plan(T, K, N, r, n);
  const LoraLayout L = lora_layout(q, T, r);
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
  p.splits = q.splits;
  p.slices = q.slices;
  p.chunk = q.chunk;
  if (q.scan) return products<true>(p, q, y_f32, s);
  const size_t smem = static_cast<size_t>(n + 1) * 4;
  cudaError_t e = allow_smem(lora_plan_kernel, smem);
  if (e == cudaSuccess) e = launch_kernel(lora_plan_kernel, dim3(1), dim3(1024), smem, s, p, q.tile_rows);
  if (e != cudaSuccess) return e;
  return q.wide ? products_wide(p, q, y_f32, s) : products<false>(p, q, y_f32, s);
}

}  // namespace moe
