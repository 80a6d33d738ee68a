// Low-rank adapters of many requests beside a shared projection (moe_lora):
//
//   y[t] = base[t] + scales[a] (x[t] A_a^T) B_a^T,   a = ids[t]
//
// Rows are taken in tiles of one adapter each.  Up to kLoraScanRows rows a CTA finds its
// tile in the ids by itself (every sixteenth row of an adapter, from its first on, has one: its
// own and the next fifteen); beyond, a launch sorts the rows by adapter and lists the tiles.  Then two launches: lora_shrink, v = x A^T as fp32 planes over slices of K, and
// lora_expand, which adds the planes in order and multiplies by B (few rows and small adapters:
// both in one).
//
// A few rows to an adapter: both products are mma.sync on operands that go from global
// memory straight to the registers that multiply them: A and B are row after row of the
// reduction dimension, as are x and v, and since a sum may take its terms in any order, a
// thread's four-byte pieces of a 32-wide step are taken from the 16 bytes that it loads.  The
// adapters' bytes are the bound.  Many rows: tcgen05 (below), x and y are.
//
// Measured (one GB300, inputs rotated so that they come from HBM): one row, 2048 x 2048, rank
// 16 4.0 us; 61 rows of 40 adapters, 4096 x 4096, rank 64 11.8 us (33 MB in 4.9 at a copy's rate;
// two launches, each three dependent trips to memory); 2000 rows of 4 requests, 2048 x 4224,
// rank 24, fp32 26.4 us (11.3); 8192 rows of 12, 8192 x 8192, rank 64 91 us (428 MB in 63).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "moe_internal.h"
#include "sm103_ptx.cuh"
#include "stream_sm103.cuh"

namespace moe {
namespace {

constexpr int kLoraScanRows = 64;
constexpr int kLoraWarps = 8;
constexpr int kRankSlice = 64;  // columns of v that one warp holds sums of

struct LoraTile {
  int adapter;  // kNoAdapter, or kNoTile: past the last tile
  int count;
};
constexpr int kNoAdapter = -1, kNoTile = -2;

struct LoraParams {
  const __nv_bfloat16 *x, *A, *B;
  const int32_t* ids;
  const float* scales;
  const void* base;
  void* y;
  float* planes;  // [splits, T, r]
  int32_t* order;  // rows of each tile (tile_rows places of a tile; -1: none)
  LoraTile* tiles;
  int32_t* err;
  int T, K, N, r, n;
  int tile_rows, max_tiles;
  int splits;  // of K (and planes, where the slices are not added at once)
  int slices;  // of r
  int chunk;   // columns of y a CTA takes, a multiple of 128 bytes (few rows: of 256 columns)
};

// ------------------------------------------------------------------- plan
// One CTA: rows counted by adapter, each adapter's first tile, rows to their tiles (in any
// order inside an adapter: what a row gets does not depend on the rows beside it).  Up to
// kPlanRows rows a thread keeps its rows' adapters and ranks; more rows are counted twice.
constexpr int kPlanThreads = 1024, kPlanEach = 8, kPlanRows = kPlanThreads * kPlanEach;
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ int32_t bins[];  // n + 1 counts, then first (next free) places in order
  __shared__ int warp_sum[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nb = p.n + 1, R = p.tile_rows;
  for (int i = tid; i < nb; i += kPlanThreads) bins[i] = 0;
  // the bins of kPlanRows rows (-1: no row), all loads under way at a time
  int b[kPlanEach], at[kPlanEach];
  auto load = [&](long long t0) {
#pragma unroll
    for (int i = 0; i < kPlanEach; ++i) {
      const long long t = t0 + tid + kPlanThreads * i;
      b[i] = -1;
      if (t < p.T) {
        const int id = p.ids[t];
        b[i] = static_cast<unsigned>(id) < static_cast<unsigned>(p.n) ? id : p.n;
      }
    }
  };
  // at[i]: place of a row in its bin.  A request's rows lie together: one atomic for a warp
  // whose rows have one adapter.
  auto take = [&](long long t0) {
#pragma unroll
    for (int i = 0; i < kPlanEach; ++i) {
      if (t0 + kPlanThreads * i >= p.T) break;
      const unsigned mask = __ballot_sync(0xffffffffu, b[i] >= 0);
      const int first = __shfl_sync(0xffffffffu, b[i], 0);
      if (__all_sync(0xffffffffu, b[i] == first || b[i] < 0)) {
        int a = 0;
        if (lane == 0 && first >= 0) a = atomicAdd(&bins[first], __popc(mask));
        at[i] = __shfl_sync(0xffffffffu, a, 0) + __popc(mask & ((1u << lane) - 1u));
      } else if (b[i] >= 0) {
        at[i] = atomicAdd(&bins[b[i]], 1);
      }
    }
  };
  load(0);
  __syncthreads();
  take(0);
  for (long long t = kPlanRows; t < p.T; t += kPlanRows) {
    load(t);
    take(t);
  }
  __syncthreads();
  // exclusive sums of the adapters' tiles, a run of adapters a thread
  const int per = (nb + kPlanThreads - 1) / kPlanThreads, b0 = min(nb, tid * per), b1 = min(nb, b0 + per);
  int tiles = 0;
  for (int i = b0; i < b1; ++i) tiles += (bins[i] + R - 1) / R;
  int inc = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int before = warp_sum[lane], all = before;
  if (lane >= warp) before = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  int tile = before + inc - tiles;
  for (int i = b0; i < b1; ++i) {
    const int c = bins[i];
    bins[i] = tile * R;
    for (int r = 0; r < c; r += R, ++tile) p.tiles[tile] = LoraTile{i < p.n ? i : kNoAdapter, min(R, c - r)};
  }
  for (int i = all + tid; i < p.max_tiles; i += kPlanThreads) p.tiles[i] = LoraTile{kNoTile, 0};
  for (int i = tid; i < all * (R / 4); i += kPlanThreads) reinterpret_cast<int4*>(p.order)[i] = make_int4(-1, -1, -1, -1);
  __syncthreads();
  if (p.T <= kPlanRows) {
#pragma unroll
    for (int i = 0; i < kPlanEach; ++i)
      if (b[i] >= 0) p.order[bins[b[i]] + at[i]] = tid + kPlanThreads * i;
    return;
  }
  for (long long t = 0; t < p.T; t += kPlanRows) {
    load(t);
    take(t);
#pragma unroll
    for (int i = 0; i < kPlanEach; ++i)
      if (b[i] >= 0) p.order[at[i]] = static_cast<int>(t) + tid + kPlanThreads * i;
  }
}

// --------------------------------------------------------------- tile rows
// The CTA's tile: its rows' numbers in `rows`, its adapter; false when it has none.  Without a
// plan (SCAN) the tile is row b and the next fifteen rows with its adapter, where a multiple of
// sixteen go before it.  (All of an adapter's rows in one CTA, sixteen at a time: 64 rows of one
// adapter of 8192 x 8192, rank 64 29.3 us, 11.5 with tiles of sixteen.)
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
      const unsigned below = (1u << lane) - 1u, before_b = (1u << (b & 31)) - 1u;
      const int from = b < 32 ? __popc(m0 & before_b) : __popc(m0) + __popc(m1 & before_b);
      const int r0 = __popc(m0 & below) - from, r1 = __popc(m0) + __popc(m1 & below) - from;
      if (i0 == mine && r0 >= 0 && r0 < 16) rows[r0] = lane;
      if (i1 == mine && r1 >= 0 && r1 < 16) rows[r1] = lane + 32;
      if (lane == 0) {
        count_slot[0] = from % 16 == 0 ? min(16, __popc(m0) + __popc(m1) - from) : 0;
        count_slot[1] = mine;
      }
    }
    __syncthreads();
    count = count_slot[0];
    adapter = count_slot[1];
    return count > 0;
  }
  const LoraTile t = p.tiles[b];
  adapter = t.adapter;
  count = t.count;
  if (threadIdx.x < 16) rows[threadIdx.x] = p.order[16 * static_cast<size_t>(b) + threadIdx.x];
  __syncthreads();
  return adapter != kNoTile;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
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
// of at most 64 columns, a slice of K, whose 32-wide steps its warps take in turn, two
// neighbours at a time (128 bytes of a row, all under way); their sums are added in the order
// of the warps.
template <int NT>
using ShrinkRed = float[kLoraWarps][32][4 * NT + 1];
// out(i, c, sum) for rows i < 16 of the tile and columns j0 + c, c < 8 NT, over pairs of steps
// [q0, q1); every output by one thread, behind a barrier.
template <int NT, typename Out>
__device__ __forceinline__ void shrink_rows(const LoraParams& p, const __nv_bfloat16* A, int j0, const int* rows,
                                            int count, int q0, int q1, ShrinkRed<NT>& red, const Out& out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const bool on0 = g < count, on1 = 8 + g < count;
  const __nv_bfloat16* x0 = p.x + static_cast<size_t>(on0 ? rows[g] : 0) * p.K;
  const __nv_bfloat16* x1 = p.x + static_cast<size_t>(on1 ? rows[8 + g] : 0) * p.K;
  float acc[NT][4] = {};
  constexpr int P = NT == 2 ? 2 : 1;  // pairs whose loads are under way at a time (what registers allow)
  for (int q = q0 + warp; q < q1; q += P * kLoraWarps) {
    uint4 lo[2 * P], hi[2 * P], col[2 * P][NT];
#pragma unroll
    for (int u = 0; u < 2 * P; ++u) {
      const int at = q + u / 2 * kLoraWarps, k = 64 * at + 32 * (u % 2) + 8 * tig;
      const bool in = k < p.K && at < q1;
      lo[u] = ldg16(x0 + k, in && on0);
      hi[u] = ldg16(x1 + k, in && on1);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        col[u][j] = ldg16(A + static_cast<size_t>(8 * j + g) * p.K + k, in && j0 + 8 * j < p.r);
    }
#pragma unroll
    for (int u = 0; u < 2 * P; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) step32(acc[j], lo[u], hi[u], col[u][j]);
  }
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
    out(i, c, v);
  }
}

template <int NT, bool SCAN>
__global__ void __launch_bounds__(kLoraWarps * 32, 2) lora_shrink_kernel(const LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int rows[16];
  __shared__ int slot[2];
  __shared__ ShrinkRed<NT> red;
  int adapter, count;
  if (!lora_tile<SCAN>(p, blockIdx.x, rows, slot, adapter, count) || adapter < 0) return;
  const int slice = blockIdx.y % p.slices, split = blockIdx.y / p.slices;
  const int j0 = slice * kRankSlice;
  const int pairs = (p.K + 63) / 64, q0 = static_cast<long long>(pairs) * split / p.splits,
            q1 = static_cast<long long>(pairs) * (split + 1) / p.splits;
  const __nv_bfloat16* A = p.A + (static_cast<size_t>(adapter) * p.r + j0) * p.K;
  float* plane = p.planes + static_cast<size_t>(split) * p.T * p.r;
  shrink_rows<NT>(p, A, j0, rows, count, q0, q1, red, [&](int i, int c, float v) {
    if (i < count && j0 + c < p.r) plane[static_cast<size_t>(rows[i]) * p.r + j0 + c] = v;
  });
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

// f[0..3] = v[row][j .. j + 3]: the planes added in their order, eight planes' loads at a time.
__device__ __forceinline__ void sum_planes(const LoraParams& p, int row, int j, float (&f)[4]) {
  constexpr int P = 8;
  const float* q = p.planes + static_cast<size_t>(row) * p.r + j;
  const size_t plane = static_cast<size_t>(p.T) * p.r;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = 0.0f;
  for (int s = 0; s < p.splits; s += P) {
    float4 a[P];
#pragma unroll
    for (int u = 0; u < P; ++u)
      if (s + u < p.splits) a[u] = *reinterpret_cast<const float4*>(q + (s + u) * plane);
#pragma unroll
    for (int u = 0; u < P; ++u)
      if (s + u < p.splits) {
        f[0] += a[u].x;
        f[1] += a[u].y;
        f[2] += a[u].z;
        f[3] += a[u].w;
      }
  }
}
// f as TERMS bf16 terms, two neighbours to a word; f keeps what is left.
template <int TERMS, int H>
__device__ __forceinline__ void split_terms(float (&f)[2 * H], uint32_t (&t)[TERMS][H]) {
#pragma unroll
  for (int z = 0; z < TERMS; ++z) {
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      t[z][j] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 b = __bfloat1622float2(h);
      // (past bf16's range the first term is infinite and the others are 0)
      f[2 * j] = isfinite(b.x) ? f[2 * j] - b.x : 0.0f;
      f[2 * j + 1] = isfinite(b.y) ? f[2 * j + 1] - b.y : 0.0f;
    }
  }
}

// ---------------------------------------------------- expand, a few rows to a tile
// A CTA: a tile and `chunk` columns of y, whose 32-wide blocks its warps take in turn.  v is
// kept in shared memory as TERMS bf16 terms.  The eight columns of an instruction are spread
// so that a thread's four of them hold eight neighbouring columns of y.  The first block's
// part of B is loaded before the planes are waited for: of what this launch reads only they
// come from the one before it, which itself began after all that went before.
//
// NT > 0: there is no launch before; every CTA makes v itself (ranks up to 8 NT), which takes
// less than a launch and a hand-over where A is small.
template <int TERMS, bool SCAN, typename Ty, int NT = 0>
__global__ void __launch_bounds__(kLoraWarps * 32, 2) lora_expand_kernel(const LoraParams p) {
  if (NT > 0) {
    pdl_wait();
    pdl_launch_dependents();
  }
  __shared__ int rows[16];
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
  if (!tile) return;  // (at once, to make room; a tile there is)
  const int n_first = c0 + 32 * warp;
  if (adapter >= 0) {
    if (NT == 0) load_step(n_first, 0);
    // the base, and the second block's (without v: the first one's too) rows of B, as far as L2
    if (base) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (8 * h + g < count && n_first + 8 * tig < c1) prefetch_l2(base + static_cast<size_t>(rows[8 * h + g]) * p.N + n_first + 8 * tig);
    }
    for (int n = n_first + lane + (NT > 0 ? 0 : 32 * kLoraWarps); n < min(c1, n_first + 32 * kLoraWarps + 32);
         n += 32 * kLoraWarps)
      for (int k = 0; k < p.r; k += 64) prefetch_l2(B + static_cast<size_t>(n) * p.r + k);
  }
  const float scale = p.scales && adapter >= 0 ? p.scales[adapter] : 1.0f;
  if (NT == 0) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if (adapter < 0) {
    copy_rows(base, y, rows, count, p.N, c0, c1);
    return;
  }
  constexpr int W = sizeof(Ty) / 2;  // 16-byte words of eight values
  if constexpr (NT > 0) {
    __shared__ ShrinkRed<NT> red;
    auto put = [&](int i, int c, float v) {
      v = c < p.r ? v * scale : 0.0f;  // (past the rank: 0 times an infinity of x)
#pragma unroll
      for (int z = 0; z < TERMS; ++z) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        vs[(z * 16 + i) * ld + c] = h;
        const float f = __bfloat162float(h);
        v = isfinite(f) ? v - f : 0.0f;  // (as split_terms)
      }
    };
    for (int o = threadIdx.x; o < 16 * (rp - 8 * NT); o += kLoraWarps * 32) put(o % 16, 8 * NT + o / 16, 0.0f);
    shrink_rows<NT>(p, p.A + static_cast<size_t>(adapter) * p.r * p.K, 0, rows, count, 0, (p.K + 63) / 64, red, put);
    load_step(n_first, 0);
  } else {
    for (int o = threadIdx.x; o < 4 * rp; o += kLoraWarps * 32) {
      const int i = o / (rp / 4), j = o % (rp / 4) * 4;
      float f[4] = {};
      if (i < count && j < p.r) {
        sum_planes(p, rows[i], j, f);
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] *= scale;
      }
      uint32_t t[TERMS][2];
      split_terms<TERMS>(f, t);
#pragma unroll
      for (int z = 0; z < TERMS; ++z) *reinterpret_cast<uint2*>(vs + (z * 16 + i) * ld + j) = make_uint2(t[z][0], t[z][1]);
    }
  }
  __syncthreads();
  for (int n0 = n_first; n0 < c1; n0 += 32 * kLoraWarps) {
    const int n = n0 + 8 * tig;
    uint4 b[2][W];
    size_t at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 8 * h + g;
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
      if (8 * h + g >= count) continue;
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

// --------------------------------------------------------- many rows to a tile
// Tiles of 128 rows on the tensor cores (tcgen05): the rows of a tile, which may lie
// anywhere, come by 16-byte cp.async into the operands' swizzled layout, through rings of
// stages that eight warps fill and one of their lanes multiplies from.  Of the 8192-row case's
// 93 us: plan 5, shrink 33 (its stages at 5.3 TB/s, the hand-over between its CTAs 2), expand 50
// (its blocks as fast as HBM takes 32 KB each), the rest launches' ends and first bytes.  The same
// rings with mma.sync took 120: instructions, and their latency at 16 warps, not bytes.
//
// Both kernels take their tensor memory before they let the next launch begin (shrink) or
// wait for the one before (expand): a CTA that waits for a launch never keeps one of that
// launch from its tensor memory.
constexpr int kWideRows = 128, kWideThreads = 256, kWideStages = 4, kMaxCluster = 8;
struct WideCtl {
  uint64_t mma[kWideStages];  // a stage's products are done
  uint64_t all;
  uint32_t tmem;
  int abort;
};
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wide_begin(WideCtl* ctl, uint32_t cols) {
  if (threadIdx.x < 32) {
    tmem_alloc(&ctl->tmem, cols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWideStages; ++i) mbar_init(&ctl->mma[i], 1);
    mbar_init(&ctl->all, 1);
    ctl->abort = 0;
    fence_mbarrier_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
}
__device__ __forceinline__ void wide_end(uint32_t tmem, uint32_t cols) {
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (threadIdx.x < 32) tmem_dealloc(tmem, cols);
}
// A wait that gives up lets the others go, and is reported; every thread stays in its loop.
__device__ __forceinline__ void wide_wait(WideCtl* ctl, uint64_t* bar, uint32_t parity, int32_t* err) {
  if (mbar_wait(bar, parity, &ctl->abort)) return;
  ctl->abort = 1;
  atomicOr(err, MOE_DEV_WAIT_TIMEOUT);
}
// 1024-byte aligned start of the dynamic shared memory
__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  const uint32_t a = smem_u32(p);
  return p + (((a + 1023u) & ~1023u) - a);
}

inline __host__ __device__ int pow2_cols(int n) {
  int c = 32;
  while (c < n) c *= 2;
  return c;
}

// Shrink.  A cluster: a tile; its CTAs: slices of K, 64 of it a stage; v [128, r] in tensor
// memory.  At the end the slices' sums are added in their order through distributed shared
// memory, a part of the rows by each CTA.
struct ShrinkGeom {
  int rn;  // r, a multiple of 16
  __host__ __device__ explicit ShrinkGeom(int r) : rn((r + 15) / 16 * 16) {}
  __host__ __device__ uint32_t stage() const { return (kWideRows + rn) * 128; }
  __host__ __device__ uint32_t cols() const { return pow2_cols(rn); }
  // (the sums, rows of rn + 4 floats, fit the ring: 512 (rn + 4) <= 512 (128 + rn))
  size_t smem() const { return 1024 + kWideStages * stage(); }
};
__global__ void __launch_bounds__(kWideThreads, 2) lora_shrink_wide_kernel(const LoraParams p) {
  __shared__ WideCtl ctl;
  __shared__ int rows[kWideRows];
  extern __shared__ uint8_t raw[];
  const ShrinkGeom geom(p.r);
  wide_begin(&ctl, geom.cols());
  const uint32_t tmem = ctl.tmem;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const LoraTile tile = p.tiles[blockIdx.x];
  if (tid < kWideRows) rows[tid] = p.order[static_cast<size_t>(blockIdx.x) * kWideRows + tid];  // (of no tile: not read)
  if (tile.adapter < 0) {  // (the whole cluster)
    wide_end(tmem, geom.cols());
    return;
  }
  __syncthreads();
  uint8_t* ring = align1024(raw);
  const uint32_t base = smem_u32(ring), stage_bytes = geom.stage();
  const int steps = (p.K + 63) / 64;
  const int s0 = static_cast<long long>(steps) * blockIdx.y / p.splits,
            s1 = static_cast<long long>(steps) * (blockIdx.y + 1) / p.splits;
  // this thread's piece of 16 bytes, of rows t0, t0 + 32, ... (which agree mod 8)
  constexpr int kStep = kWideThreads / 8, kRowsEach = kWideRows / kStep;
  const int piece = tid & 7, t0 = tid >> 3;
  const uint32_t put = base + t0 * 128 + ((piece ^ (t0 & 7)) << 4);
  const __nv_bfloat16* xp[kRowsEach];
  uint32_t xbytes[kRowsEach];
#pragma unroll
  for (int i = 0; i < kRowsEach; ++i) {
    const int row = rows[t0 + kStep * i];
    xp[i] = p.x + static_cast<size_t>(max(row, 0)) * p.K + 64 * s0 + 8 * piece;
    xbytes[i] = row >= 0 ? 16u : 0u;
  }
  const size_t apitch = static_cast<size_t>(kStep) * p.K;
  const __nv_bfloat16* ap = p.A + (static_cast<size_t>(tile.adapter) * p.r + t0) * p.K + 64 * s0 + 8 * piece;
  int k = 64 * s0 + 8 * piece, left = s1 - s0;  // of the next stage to be filled; those left
  uint32_t slot = 0;
  auto load = [&]() {
    if (left > 0) {
      const uint32_t to = put + slot * stage_bytes;
      const bool in = k < p.K;  // (past it nothing is read: K is a multiple of a piece)
#pragma unroll
      for (int i = 0; i < kRowsEach; ++i) {
        cp_async_16(to + i * kStep * 128, in ? xp[i] : p.x, in ? xbytes[i] : 0u);
        xp[i] += 64;
      }
      const __nv_bfloat16* a = ap;
      for (int j = t0; j < geom.rn; j += kStep, a += apitch) {
        const bool on = in && j < p.r;
        cp_async_16(to + (kWideRows + j - t0) * 128, on ? a : p.x, on ? 16u : 0u);
      }
      ap += 64;
      k += 64;
      --left;
      slot = slot + 1 == kWideStages ? 0 : slot + 1;
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kWideStages; ++i) load();
  const uint32_t idesc = make_idesc_bf16_f32(kWideRows, geom.rn, 0, 0);
  for (int i = 0; i < s1 - s0; ++i) {
    if (i == 0)
      cp_wait<kWideStages - 1>();
    else
      cp_wait<kWideStages - 2>();
    fence_proxy_async_smem();
    __syncthreads();  // the stage is there
    if (tid == 0) {
      tc_fence_after_sync();
      const uint32_t at = base + static_cast<uint32_t>(i % kWideStages) * stage_bytes;
      const uint64_t xd = make_smem_desc_sw128(at, 16, 1024), ad = make_smem_desc_sw128(at + kWideRows * 128, 16, 1024);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        tc_mma_f16(tmem, smem_desc_advance(xd, 32 * q), smem_desc_advance(ad, 32 * q), idesc, (i | q) != 0);
      tc_commit(&ctl.mma[i % kWideStages]);
      if (i + 1 == s1 - s0) tc_commit(&ctl.all);
    }
    // the stage that is filled next was multiplied from one step before
    if (i > 0) {
      wide_wait(&ctl, &ctl.mma[(i - 1) % kWideStages], ((i - 1) / kWideStages) & 1, p.err);
      load();
    }
  }
  wide_wait(&ctl, &ctl.all, 0, p.err);
  __syncwarp();
  tc_fence_after_sync();
  const int mine = 32 * (warp & 3) + lane;  // this thread's row; every second 32 of its columns
  const bool alone = p.splits == 1;
  float* part = reinterpret_cast<float*>(ring);
  float* to = alone ? p.planes + static_cast<size_t>(max(rows[mine], 0)) * p.r : part + mine * (geom.rn + 4);
  const int upto = !alone ? geom.rn : rows[mine] >= 0 ? p.r : 0;
  for (int c = 32 * (warp >> 2); c < geom.rn; c += 64) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c, v);
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      if (c + j < upto) *reinterpret_cast<uint4*>(to + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  }
  if (!alone) {
    __syncwarp();
    cluster_sync();
    const int each = (kWideRows + p.splits - 1) / p.splits, first = each * blockIdx.y, quads = p.r / 4;
    for (int o = tid; o < each * quads; o += kWideThreads) {
      const int t = first + o / quads, c = 4 * (o % quads);
      if (t >= kWideRows || rows[t] < 0) continue;
      const float* at = part + t * (geom.rn + 4) + c;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int z = 0; z < p.splits; ++z) {
        const float4 w = ld_cluster_v4(mapa_shared(at, z));
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      *reinterpret_cast<float4*>(p.planes + static_cast<size_t>(rows[t]) * p.r + c) = v;
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves before its sums are read
  }
  wide_end(tmem, geom.cols());
}

// Expand.  A CTA: a tile and `chunk` columns of y in blocks of 128 bytes of a row of y.  v's
// bf16 terms lie in tensor memory as the operand that stays; a stage holds the block's rows
// of B and the tile's base; a block's products go to one of two sums in tensor memory and
// are finished while the next block's are made: sums and base are added in place of the base
// in shared memory, and go from there to y by whole rows of 128 bytes.  Two warps have 32 rows
// of a tile to themselves: each brings and stores 16 of them and adds half of the columns of
// all, so that they wait for one another once a block, and for the others for B alone.
template <typename Ty>
struct ExpandGeom {
  static constexpr int TERMS = sizeof(Ty) == 2 ? 2 : 3;
  static constexpr int COLS = 128 / sizeof(Ty);
  int atoms;  // of 64 of the rank
  int ksteps; // of 16 of the rank
  int kcols;  // tensor-memory columns of a term, whole stores of 16
  __host__ __device__ explicit ExpandGeom(int r) : atoms((r + 63) / 64), ksteps((r + 15) / 16), kcols((r + 31) / 32 * 16) {}
  __host__ __device__ uint32_t stage() const { return (atoms * COLS + kWideRows) * 128; }
  __host__ __device__ uint32_t sums() const { return TERMS * kcols; }
  __host__ __device__ uint32_t cols() const { return pow2_cols(TERMS * kcols + 2 * COLS); }
  size_t smem() const { return 1024 + kWideStages * stage(); }
};
template <typename Ty>
__global__ void __launch_bounds__(kWideThreads, 2) lora_expand_wide_kernel(const LoraParams p) {
  using Geom = ExpandGeom<Ty>;
  constexpr int TERMS = Geom::TERMS, COLS = Geom::COLS, V = 16 / sizeof(Ty);
  __shared__ WideCtl ctl;
  __shared__ int rows[kWideRows];
  extern __shared__ uint8_t raw[];
  const Geom geom(p.r);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const LoraTile tile = p.tiles[blockIdx.x];
  if (tid < kWideRows) rows[tid] = p.order[static_cast<size_t>(blockIdx.x) * kWideRows + tid];
  if (tile.adapter == kNoTile) return;  // (at once, to make room; a tile there is)
  const float scale = p.scales && tile.adapter >= 0 ? p.scales[tile.adapter] : 1.0f;
  wide_begin(&ctl, geom.cols());
  const uint32_t tmem = ctl.tmem;
  const int c0 = blockIdx.y * p.chunk, c1 = min(p.N, c0 + p.chunk), blocks = (c1 - c0 + COLS - 1) / COLS;
  const Ty* base = static_cast<const Ty*>(p.base);
  Ty* y = static_cast<Ty*>(p.y);
  uint8_t* ring = align1024(raw);
  const uint32_t ring_at = smem_u32(ring), stage_bytes = geom.stage(), base_at = geom.atoms * COLS * 128;
  // B's pieces of 16 bytes: eight threads to a row, kStep rows at a time
  constexpr int kStep = kWideThreads / 8;
  const int bpiece = tid & 7, t0 = tid >> 3;
  const uint32_t bput = ring_at + t0 * 128 + ((bpiece ^ (t0 & 7)) << 4);
  // the base's and y's: eight lanes to a row, four rows at a time of the warp's sixteen
  const int quarter = warp & 3, half = warp >> 2, piece = lane & 7;
  const int wrow = 32 * quarter + 16 * half + (lane >> 3);  // + 4 i
  auto place = [&](int i) { return (wrow + 4 * i) * 128 + ((piece ^ (lane >> 3) ^ (4 * (i & 1))) << 4); };
  const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
  const uint32_t idesc = make_idesc_bf16_f32(kWideRows, COLS, 0, 0);
  const __nv_bfloat16* bp =
      p.B + (static_cast<size_t>(max(tile.adapter, 0)) * p.N + c0 + t0) * p.r + 8 * bpiece;
  size_t off[4];
  uint32_t ybytes[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = rows[wrow + 4 * i];
    off[i] = static_cast<size_t>(max(row, 0)) * p.N + c0 + V * piece;
    ybytes[i] = row >= 0 ? 16u : 0u;
  }
  int n_load = 0, left = blocks;  // columns of the next block to be brought, from c0; blocks left
  uint32_t slot = 0;
  auto load = [&]() {
    if (left > 0) {
      const uint32_t at = slot * stage_bytes;
      for (int a = 0; a < geom.atoms; ++a)
#pragma unroll
        for (int i = 0; i < COLS / kStep; ++i) {
          const bool on = c0 + n_load + t0 + kStep * i < p.N && 64 * a + 8 * bpiece < p.r;
          cp_async_16(bput + at + (a * COLS + kStep * i) * 128, on ? bp + static_cast<size_t>(kStep * i) * p.r + 64 * a : p.B,
                      on ? 16u : 0u);
        }
      bp += static_cast<size_t>(COLS) * p.r;
      if (base) {
        const bool in = c0 + n_load + V * piece < p.N;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          cp_async_16(ring_at + at + base_at + place(i), in ? base + off[i] + n_load : base, in ? ybytes[i] : 0u);
      }
      n_load += COLS;
      --left;
      slot = slot + 1 == kWideStages ? 0 : slot + 1;
    }
    cp_commit();
  };
  if (tile.adapter >= 0) {  // nothing of these comes from the launch before (the planes do)
#pragma unroll
    for (int i = 0; i < kWideStages; ++i) load();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (tile.adapter < 0) {
    copy_rows(base, y, rows, tile.count, p.N, c0, c1);
    wide_end(tmem, geom.cols());
    return;
  }
  {
    // a row of v by two threads, 32 of the rank (16 columns) at a time
    const int row = rows[32 * quarter + lane];
    for (int j = 32 * half; j < 2 * geom.kcols; j += 64) {
      float f[4][8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool on = row >= 0 && j + 8 * q < p.r;
        const float4* at = reinterpret_cast<const float4*>(p.planes + static_cast<size_t>(max(row, 0)) * p.r + j + 8 * q);
        const float4 a = on ? at[0] : make_float4(0.f, 0.f, 0.f, 0.f), b = on ? at[1] : make_float4(0.f, 0.f, 0.f, 0.f);
        f[q][0] = a.x, f[q][1] = a.y, f[q][2] = a.z, f[q][3] = a.w, f[q][4] = b.x, f[q][5] = b.y, f[q][6] = b.z, f[q][7] = b.w;
      }
      uint32_t t[TERMS][16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[q][i] *= scale;
        uint32_t u[TERMS][4];
        split_terms<TERMS>(f[q], u);
#pragma unroll
        for (int z = 0; z < TERMS; ++z)
#pragma unroll
          for (int i = 0; i < 4; ++i) t[z][4 * q + i] = u[z][i];
      }
#pragma unroll
      for (int z = 0; z < TERMS; ++z) tmem_st_32x32b_x16(lanes + z * geom.kcols + j / 2, t[z]);
    }
    tc_wait_st();
  }
  for (int b = 0; b <= blocks; ++b) {
    if (b < blocks) {
      cp_wait<kWideStages - 2>();
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncthreads();  // the stage (and, at first, v) is there, the sums' former block is finished
      if (warp == 0) {
        tc_fence_after_sync();
        const uint32_t from = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t bd = make_smem_desc_sw128(ring_at + static_cast<uint32_t>(b % kWideStages) * stage_bytes, 16, 1024);
        const uint32_t to = from + geom.sums() + (b & 1) * COLS;
        for (int z = 0; z < TERMS; ++z)
          for (int k = 0; k < geom.ksteps; ++k)
            tc_mma_f16_ts_elect(to, from + z * geom.kcols + 8 * k,
                                smem_desc_advance(bd, (k >> 2) * COLS * 128 + (k & 3) * 32), idesc, (z | k) != 0);
        tc_commit_elect(&ctl.mma[b % kWideStages]);
        __syncwarp();
      }
    }
    if (b == 0) continue;
    const int f = b - 1;  // the block that is finished now
    wide_wait(&ctl, &ctl.mma[f % kWideStages], (f / kWideStages) & 1, p.err);
    __syncwarp();
    tc_fence_after_sync();
    uint8_t* tile_at = ring + static_cast<size_t>(f % kWideStages) * stage_bytes + base_at;
    uint8_t* mine = tile_at + (32 * quarter + lane) * 128;
    constexpr int MINE = COLS / 2;  // columns
    uint32_t v[MINE];
    if constexpr (MINE == 32)
      tmem_ld_32x32b_x32(lanes + geom.sums() + (f & 1) * COLS + MINE * half, v);
    else
      tmem_ld_32x32b_x16(lanes + geom.sums() + (f & 1) * COLS + MINE * half, v);
    uint4 w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = base ? *reinterpret_cast<const uint4*>(mine + (((4 * half + q) ^ (lane & 7)) << 4)) : make_uint4(0u, 0u, 0u, 0u);
    tc_wait_ld();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t u[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(Ty) == 2) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(
              __uint_as_float(v[8 * q + 2 * i]) + __uint_as_float(u[i] << 16),
              __uint_as_float(v[8 * q + 2 * i + 1]) + __uint_as_float(u[i] & 0xffff0000u));
          u[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          u[i] = __float_as_uint(__uint_as_float(v[4 * q + i]) + __uint_as_float(u[i]));
        }
      }
      *reinterpret_cast<uint4*>(mine + (((4 * half + q) ^ (lane & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    named_bar_sync(1 + quarter, 64);  // the other half of the columns
    const int n = f * COLS;
    const bool in = c0 + n + V * piece < c1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 out = *reinterpret_cast<const uint4*>(tile_at + place(i));
      if (in && ybytes[i]) *reinterpret_cast<uint4*>(y + off[i] + n) = out;
    }
    __syncwarp();  // (the warp's rows of the stage are filled again)
    load();
  }
  wide_end(tmem, geom.cols());
}

constexpr int kSms = 152;  // a constant: results must not depend on the device

// How T rows of n adapters are taken: `scan`, tiles found by the CTAs themselves; `at_once`,
// these in one launch; `wide`, the kernels for many rows to a tile.
struct LoraPlan {
  bool scan, at_once, wide;
  int tile_rows, tiles, slices, splits, chunk;
};
// Rows from which n adapters are taken by the kernels for many rows to a tile: 1024, and 64 an
// adapter, or 32 from 2048 on.
// (measured, 4096 x 4096, rank 64, rows in any order, us of few-row : many-row kernels: 1024 rows
// of 16 adapters 23.7 : 21.7, of 32 27.2 : 32.0; 4096 of 128 107 : 96, of 256 119 : 131; 256 of 4
// 13.2 : 17.5.  The rule does not look at K, N and r.  What the switch does at other sizes, requests
// in runs, us of 1023 : 1024 rows: 2048 x 2048 one adapter, rank 16 14.3 : 13.4, rank 256 36 : 30, 16
// adapters 12.3 : 14.6 and 30 : 39; 8192 x 8192 one adapter 27.9 : 24.3 and 88 : 47, 16 adapters 33 : 27
// and 106 : 74.  So wide projections and large ranks would gain from a switch at fewer rows, and small
// ones with many adapters from one at more)
long long lora_wide_from(int n) { return n < 32 ? std::max(1024ll, 64ll * n) : std::max(2048ll, 32ll * n); }

LoraPlan lora_plan(int T, int K, int N, int r, int n, bool y_f32) {
  LoraPlan q{};
  q.scan = T <= kLoraScanRows;
  q.wide = T >= lora_wide_from(n);
  q.tile_rows = q.wide ? kWideRows : 16;
  q.tiles = q.scan ? T : static_cast<int>(std::min<long long>(T, (T + q.tile_rows - 1ll) / q.tile_rows + n));
  // one launch instead of two, where every CTA of 256 columns makes v again: as long on the GPU (us of two : of one, 1, 16, 32, 64 rows with
  // adapters of their own: 2048 x 2048, rank 16 5.1 : 4.7, 5.5 : 5.1, 6.1 : 6.1, 7.1 : 7.2; 4096 x
  // 4096, rank 16 5.1 : 6.1, 6.0 : 7.6, 7.1 : 8.7, 8.2 : 9.7), and 1.5 less of the caller's time
  q.at_once = T <= 32 && r <= 32 && static_cast<long long>(r) * K <= 32768;
  // adapters that some row has, about, and tiles
  const long long used = std::min<long long>(T, static_cast<long long>(n) * T / std::max(1, T + n / 2));
  const long long tiles =
      std::max(1ll, q.scan ? used * ((T + 16 * used - 1) / std::max(1ll, 16 * used))
                           : q.wide ? (T + q.tile_rows - 1) / q.tile_rows + n / 2 : used + T / 32);
  q.slices = q.wide ? 1 : (r + kRankSlice - 1) / kRankSlice;
  // slices of K: as many CTAs as have room at a time (two an SM)
  const long long room = std::max(1ll, 2ll * kSms / (tiles * q.slices));
  if (q.wide) {  // of four stages at least
    q.splits = static_cast<int>(std::min<long long>({room, (K + 255) / 256, kMaxCluster}));
  } else {  // and no more than what its warps load at once need (two steps each)
    const int pairs = (K + 63) / 64;
    const long long most = std::min<long long>(room, (pairs + kLoraWarps - 1) / kLoraWarps);
    const long long rounds = ((pairs + most - 1) / most + kLoraWarps - 1) / kLoraWarps;
    q.splits = static_cast<int>((pairs + rounds * kLoraWarps - 1) / (rounds * kLoraWarps));
  }
  // y's columns: as many CTAs as have room, in blocks of 128 bytes, or of 32 columns for each warp
  // (fp32 in blocks of 64 columns, 320 to a CTA instead of 288: 2000 rows of 4 28.2 us, not 27.4)
  const int unit = !q.wide ? 32 * kLoraWarps : y_f32 ? 32 : 64, units = (N + unit - 1) / unit;
  const int chunks = static_cast<int>(std::min<long long>(std::max(1ll, 2ll * kSms / tiles), units));
  q.chunk = (units + chunks - 1) / chunks * unit;
  return q;
}

struct LoraLayout {
  size_t planes, order, tiles, total;
};
LoraLayout lora_layout(const LoraPlan& q, int T, int r) {
  LoraLayout L{};
  size_t cur = sizeof(ControlBlock);
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur = (cur + bytes + 255) / 256 * 256;
    return o;
  };
  if (!q.at_once) L.planes = take(static_cast<size_t>(q.wide ? 1 : q.splits) * T * r * 4);
  if (!q.scan) {
    L.order = take(static_cast<size_t>(q.tiles) * q.tile_rows * 4);
    L.tiles = take(static_cast<size_t>(q.tiles) * sizeof(LoraTile));
  }
  L.total = cur;
  return L;
}

// Once a kernel and device: all the shared memory that any of its launches takes.
template <auto KERNEL>
cudaError_t allow_smem(size_t most) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_relaxed))) return e;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
  if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

size_t expand_smem(const LoraParams& p, bool y_f32) {
  return static_cast<size_t>(y_f32 ? 3 : 2) * 16 * ((p.r + 31) / 32 * 32 + 8) * 2;
}
template <bool SCAN>
cudaError_t products(const LoraParams& p, const LoraPlan& q, bool y_f32, cudaStream_t s) {
  const dim3 block(kLoraWarps * 32), grid(q.tiles, p.splits * p.slices), egrid(q.tiles, (p.N + p.chunk - 1) / p.chunk);
  auto shrink = p.r <= 16 ? lora_shrink_kernel<2, SCAN> : p.r <= 32 ? lora_shrink_kernel<4, SCAN> : lora_shrink_kernel<8, SCAN>;
  cudaError_t e = launch_kernel(shrink, grid, block, 0, s, p);
  if (e != cudaSuccess) return e;
  auto expand = y_f32 ? lora_expand_kernel<3, SCAN, float> : lora_expand_kernel<2, SCAN, __nv_bfloat16>;
  e = launch_kernel(expand, egrid, block, expand_smem(p, y_f32), s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}
// Both products in one launch (few rows, small adapters).
template <int NT>
cudaError_t products_at_once(const LoraParams& p, const LoraPlan& q, bool y_f32, cudaStream_t s) {
  auto kern = y_f32 ? lora_expand_kernel<3, true, float, NT> : lora_expand_kernel<2, true, __nv_bfloat16, NT>;
  const cudaError_t e = launch_kernel(kern, dim3(q.tiles, (p.N + p.chunk - 1) / p.chunk), dim3(kLoraWarps * 32),
                                      expand_smem(p, y_f32), s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename Ty>
cudaError_t expand_wide(const LoraParams& p, cudaStream_t s) {
  const ExpandGeom<Ty> geom(p.r);
  const cudaError_t e = allow_smem<lora_expand_wide_kernel<Ty>>(ExpandGeom<Ty>(kLoraMaxRank).smem());
  if (e != cudaSuccess) return e;
  const dim3 grid(p.max_tiles, (p.N + p.chunk - 1) / p.chunk);
  return launch_kernel(lora_expand_wide_kernel<Ty>, grid, dim3(kWideThreads), geom.smem(), s, p);
}
cudaError_t products_wide(const LoraParams& p, const LoraPlan& q, bool y_f32, cudaStream_t s) {
  const size_t shrink = ShrinkGeom(p.r).smem();
  cudaError_t e = allow_smem<lora_shrink_wide_kernel>(ShrinkGeom(kLoraMaxRank).smem());
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = p.splits;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = g_pdl ? 1 : 0;
  cfg.gridDim = dim3(q.tiles, p.splits);
  cfg.blockDim = dim3(kWideThreads);
  cfg.dynamicSmemBytes = shrink;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, lora_shrink_wide_kernel, p);
  if (e != cudaSuccess) return e;
  e = y_f32 ? expand_wide<float>(p, s) : expand_wide<__nv_bfloat16>(p, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t lora_need_bytes(int T, int K, int N, int r, int n) {
  return lora_layout(lora_plan(T, K, N, r, n, false), T, r).total;  // (y's type is that of the chunk alone)
}

// The most that T rows or fewer need.  A batch of the few-row kernels can need more than a
// larger one: many rows have one plane, few rows one for each slice of K, whose number falls as
// the tiles become more.  With a plan the tiles grow with T, so from the first T on that has a
// single slice the need grows too, up to the last T of those kernels.
size_t lora_workspace_bytes(int T, int K, int N, int r, int n) {
  const int few = std::min<long long>(T, lora_wide_from(n) - 1);
  size_t most = std::max(lora_need_bytes(T, K, N, r, n), lora_need_bytes(few, K, N, r, n));
  for (int t = 1; t < few; ++t) {
    const LoraPlan q = lora_plan(t, K, N, r, n, false);
    if (!q.scan && q.splits == 1) break;
    most = std::max(most, lora_layout(q, t, r).total);
  }
  return most;
}

cudaError_t launch_lora(int T, int K, int N, int r, int n, const void* x, const int32_t* ids, const void* A,
                        const void* B, const float* scales, const void* base, void* y, bool y_f32, uint8_t* ws,
                        cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  const LoraPlan q = lora_plan(T, K, N, r, n, y_f32);
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
  p.err = &reinterpret_cast<ControlBlock*>(ws)->err;
  p.T = T;
  p.K = K;
  p.N = N;
  p.r = r;
  p.n = n;
  p.tile_rows = q.tile_rows;
  p.max_tiles = q.tiles;
  p.splits = q.splits;
  p.slices = q.slices;
  p.chunk = q.chunk;
  if (q.at_once) return r <= 16 ? products_at_once<2>(p, q, y_f32, s) : products_at_once<4>(p, q, y_f32, s);
  if (q.scan) return products<true>(p, q, y_f32, s);
  const size_t smem = static_cast<size_t>(n + 1) * 4;
  cudaError_t e = allow_smem<lora_plan_kernel>(static_cast<size_t>(kLoraMaxAdapters + 1) * 4);
  if (e == cudaSuccess) e = launch_kernel(lora_plan_kernel, dim3(1), dim3(kPlanThreads), smem, s, p);
  if (e != cudaSuccess) return e;
  return q.wide ? products_wide(p, q, y_f32, s) : products<false>(p, q, y_f32, s);
}

}  // namespace moe
