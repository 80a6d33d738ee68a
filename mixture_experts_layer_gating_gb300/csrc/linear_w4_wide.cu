// moe_linear_w4 for many rows (linear_w4_wide() says when): the same runs of
// stages over the CTAs as for fewer rows, the products on tcgen05.
//
//   y[m][n] = sum over groups q of s[n][q] * (sum over the group's k of
//             (code[n][k] - zero[n][q]) * x[m][k])
//
// mma.sync takes 8 tensor cycles for 256 weights and 8 rows: at 32 rows more than
// the weights take from HBM (58 us against 40 for 4096 x 131072), beside the loads
// of the token rows into every warp's registers.  tcgen05 takes 16 cycles for 128
// weight rows x 16 k x 32 token rows.  The weights are its operand in tensor
// memory: a thread takes one weight row's codes from the stage, makes them bf16
// (code - zero, exact) in registers and stores them there, so that nothing is
// expanded into shared memory.  A group's sums come back to the thread of the
// weight row, which multiplies them by the group's scale and adds in fp32.
//
// 32 rows x 4096 x 131072, fp32 out (HBM floor 42 to 47 us): groups of 128 74 us (mma.sync
// 170), of 64 77, of 32 95; with zero points 80, 88, 108.  What bounds it: eleven
// half-rate instructions for eight codes, in two converter warps a scheduler, which
// take 700 of the 1100 cycles of a unit and share the scheduler with others (adders,
// on two schedulers an issuer) in the rest: ALU pipe 49 %, issue 53 % (8192 x 32768).
//
// A stage is 256 weight rows x 256 k (32 KB) and the rows' 256 k (16 KB: read
// once for 256 weight rows, or they would cost as many bytes from L2 as the
// weights from HBM).  Roles:
//   converters (two warpgroups, 128 weight rows each): codes -> tensor memory, a
//     unit of 128 or 64 k at a time, into one of two to four buffers (three of 128 k:
//     74 us, two: 93);
//   issuers (a warp for each half): the products of a unit, into one of two sets of
//     sums;
//   adders (two warpgroups): a unit's sums times their scales, in registers;
//   finisher (a warp): a whole strip's sums to y;
//   producer: TMA.
#include "linear_w4.cuh"

namespace moe {

namespace {

constexpr int kWideTokens = 32;  // rows of x in a stage (zeros beyond M)
constexpr int kWideWeights = kWideStrip * 128;
constexpr int kWideSlot = kWideWeights + kWideTokens * 512;
// warps of the roles: converters 0 - 7, adders 8 - 15, finisher, producer, issuers
constexpr int kWideAdders = 256, kWideAdd = 256, kWideFinish = 512, kWideProduce = 544, kWideIssue = 576, kWideBlock = 640;

constexpr int kWideMaxUnits = 4;
struct WideCtrl {
  StreamRing ring;
  uint64_t ready[kWideMaxUnits], done[kWideMaxUnits];  // a buffer's weights are there, are multiplied
  uint64_t sums[kWideMaxUnits], read[kWideMaxUnits];   // a set of sums is there, is read
  uint64_t red_full, red_empty;  // a strip's sums
  uint64_t drain;
  uint32_t tmem;
};
constexpr int kWideRed = kWideTokens * kWideStrip * 4;
constexpr int kWideStages = (kStreamSmemMax - 1024 - kWideRed - static_cast<int>(sizeof(WideCtrl))) / kWideSlot;
constexpr int kWideBytes = 1024 + kWideStages * kWideSlot + kWideRed + static_cast<int>(sizeof(WideCtrl));
static_assert(kWideStages >= 3 && kWideStages <= kMaxStages && kWideSlot % 1024 == 0, "ring");

// x in the order of the codes' pairs (a word's codes e and e + 4 side by side),
// padded with zeros to whole stages: eight inputs a thread.
__global__ void __launch_bounds__(256) linear_w4_order_kernel(const __grid_constant__ LinParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int k0 = (blockIdx.x * 256 + threadIdx.x) * 8, row = blockIdx.y;
  if (k0 >= p.Kp) return;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (k0 < p.K) x = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(row) * p.K + k0));
  uint4 v;
  v.x = __byte_perm(x.x, x.z, 0x5410);
  v.y = __byte_perm(x.x, x.z, 0x7632);
  v.z = __byte_perm(x.y, x.w, 0x5410);
  v.w = __byte_perm(x.y, x.w, 0x7632);
  *reinterpret_cast<uint4*>(p.xp + static_cast<size_t>(row) * p.Kp + k0) = v;
}

__device__ __forceinline__ void prefetch_row(const void* p, size_t bytes) {
  const uint8_t* at = static_cast<const uint8_t*>(p);
  for (size_t i = 0; i < bytes; i += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i));
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at + bytes - 1));
}

// Eight groups' scales (or zeros) of a weight row from group q0 (a multiple of
// eight) on; those beyond the row's last are 0.  A warp's 32 rows lie in 32
// sectors: a load for each unit and group would cost more than the products.
struct WideScales {
  uint32_t v[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* sc, int N, int groups, int n, int q0) {
    v[0] = v[1] = v[2] = v[3] = 0;
    const size_t at = static_cast<size_t>(n) * groups + q0;
    const bool wide = (groups & 7) == 0;
    // (predicated, not in a branch, whose end would wait for it; for the zeros, which the
    // converters load, that gains nothing: 86 us either way in groups of 64, 83 for 79 in
    // groups of 128)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3])
        : "l"(sc + at), "r"(static_cast<uint32_t>(wide && n < N)));
    if (!wide && n < N) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (q0 + i < groups)
          v[i >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(sc) + at + i)) << (16 * (i & 1));
    }
  }
  __device__ __forceinline__ float get(int i) const {  // (selects, not an array in memory)
    const uint32_t a = i & 4 ? v[2] : v[0], b = i & 4 ? v[3] : v[1], w = i & 2 ? b : a;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};
struct WideZeros {
  uint32_t v[2];
  __device__ __forceinline__ void load(const uint8_t* zp, int N, int groups, int n, int q0) {
    v[0] = v[1] = 0;
    if (n >= N) return;
    const size_t at = static_cast<size_t>(n) * groups + q0;
    if ((groups & 7) == 0 && (reinterpret_cast<uintptr_t>(zp) & 7) == 0) {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(zp + at));
      v[0] = t.x; v[1] = t.y;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (q0 + i < groups) v[i >> 2] |= static_cast<uint32_t>(__ldg(zp + at + i)) << (8 * (i & 3));
    }
  }
  // From zero i on (two in one word), zero by zero as the pair of bf16 128 + zero.
  __device__ __forceinline__ uint32_t from(int i) const { return (i & 4 ? v[1] : v[0]) >> (8 * (i & 3)); }
  static __device__ __forceinline__ uint32_t pair(uint32_t w, int h) {
    return __byte_perm(w, 0x43434343u, h ? 0x4141 : 0x4040) & 0xff0fff0fu;
  }
};

template <int GRP, bool ZERO, typename TY>
__global__ void __launch_bounds__(kWideBlock, 1)
    linear_w4_wide_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                          const __grid_constant__ LinParams p) {
  constexpr int UNIT = GRP == 32 ? 64 : 128;   // k of a unit
  // Buffers of weights (both halves': UNIT columns) and sets of sums (both halves': 64
  // columns a sum) fill the 512 columns.  Groups of 64 in units of 64 k, four and four
  // of them: 87 us, not 77, when it was tried (4096 x 131072, 32 rows).
  constexpr int NA = GRP == 128 ? 3 : GRP == 64 ? 2 : 4, ND = 2;
  constexpr int UPC = 256 / UNIT;             // units of a stage
  constexpr int SUMS = UNIT / GRP;            // groups, and sums, of a unit: 1 or 2
  constexpr int STEPS = GRP / 16;             // k16 steps of a sum
  constexpr int PER = GRP / 32;     // stages of eight groups
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* red = reinterpret_cast<float*>(ring + kWideStages * kWideSlot);
  auto* ctl = reinterpret_cast<WideCtrl*>(ring + kWideStages * kWideSlot + kWideRed);
  StreamRing* sr = &ctl->ring;
  const int tid = threadIdx.x, b = blockIdx.x, lane = tid & 31;
  const int C = p.Kp / 256, S = (p.N + kWideStrip - 1) / kWideStrip, groups = p.K / GRP;
  const Split sp = make_split(static_cast<long long>(S) * C, gridDim.x);
  const long long lo = split_lo(sp, b), hi = split_lo(sp, b + 1);

  if (tid == 0) {
    for (int i = 0; i < kWideMaxUnits; ++i) {
      mbar_init(&ctl->ready[i], 8);
      mbar_init(&ctl->done[i], 2);
      mbar_init(&ctl->sums[i], 2);
      mbar_init(&ctl->read[i], 8);
    }
    mbar_init(&ctl->red_full, 8);
    mbar_init(&ctl->red_empty, 1);
    mbar_init(&ctl->drain, 2);
    sr->init(1, 1, 2);
  }
  if (tid < 32) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_wait();
  pdl_launch_dependents();
  int s = static_cast<int>(lo / C), kc = static_cast<int>(lo % C);
  int left = static_cast<int>(hi - lo);
  const uint32_t tmem = ctl->tmem;  // buffers [NA][half][UNIT / 2 columns], sums [ND][half][SUMS][32]
  constexpr uint32_t kSums = NA * UNIT, kSet = 64 * SUMS;
  static_assert(kSums + ND * kSet <= 512, "tensor memory");
  const uint32_t lanes = static_cast<uint32_t>((tid >> 5) & 3) << 21;  // the warp's 32 lanes
  const int half = (tid >> 7) & 1, row = tid & 255;  // converters and adders: of the strip's 256 weight rows

  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (warp >= kWideIssue / 32) {
    // Issuers.  The whole warp runs this, one elected lane issues: where the compiler sees
    // one address for the warp, a product of 128 x 32 x 16 issues in 16 cycles, from a
    // single lane's branch in 51.
    constexpr uint32_t kIdesc = make_idesc_bf16_f32(128, kWideTokens, 0, 0);
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0), w = warp - kWideIssue / 32;  // w: the half
    left = __shfl_sync(0xffffffffu, left, 0);
    RingPos pos, wpos, spos;
    bool ok = true;
#pragma unroll 1
    for (; left > 0 && ok; --left) {
      ok = __all_sync(0xffffffffu, mbar_wait(&sr->full[pos.at], pos.phase, &sr->abort));
      const uint32_t x = smem_u32(ring) + pos.at * kWideSlot + kWideWeights;
#pragma unroll 1
      for (int u = 0; u < UPC && ok; ++u) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl->ready[wpos.at], wpos.phase, &sr->abort) &&
                                         mbar_wait(&ctl->read[spos.at], spos.phase ^ 1u, &sr->abort));
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t d0 = make_smem_desc_sw128(x + u * (UNIT / 64) * kWideTokens * 128, 16, 1024);
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
          for (int h = 0; h < SUMS; ++h) {
            const int k = h * STEPS + i;
            const uint64_t d = smem_desc_advance(d0, (k >> 2) * kWideTokens * 128 + (k & 3) * 32);
            tc_mma_f16_ts_elect(base + kSums + spos.at * kSet + (w * SUMS + h) * 32,
                                base + wpos.at * UNIT + w * (UNIT / 2) + k * 8, d, kIdesc, i != 0);
          }
        tc_commit_elect(&ctl->done[wpos.at]);
        tc_commit_elect(&ctl->sums[spos.at]);
        wpos.next(NA);
        spos.next(ND);
      }
      tc_commit_elect(&sr->empty[pos.at]);  // (the codes were read before the units were ready)
      pos.next(kWideStages);
    }
    if (!ok) sr->give_up(p.err);
    tc_commit_elect(&ctl->drain);  // nothing is in flight when the CTA ends
    mbar_wait_drain(&ctl->drain, 0);
    __syncwarp();
    asm volatile("bar.arrive 2, %0;" ::"n"(kWideFinish + 64) : "memory");
    return;
  }
  if (tid >= kWideProduce) {  // producer
    if (lane == 0) {
      const uint64_t once = l2_policy_evict_first(), often = l2_policy_evict_last();
      RingPos pos;
#pragma unroll 1
      for (; left > 0; --left) {
        if (!mbar_wait(&sr->empty[pos.at], pos.phase ^ 1u, &sr->abort)) {
          sr->give_up(p.err);
          break;
        }
        uint64_t* full = &sr->full[pos.at];
        uint8_t* dst = ring + pos.at * kWideSlot;
        mbar_arrive_expect_tx(full, kWideSlot);
        tma_load_2d(dst, &mw, full, kc * 128, s * kWideStrip, once);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tma_load_2d(dst + kWideWeights + i * kWideTokens * 128, &mx, full, kc * 256 + i * 64, 0, often);
        pos.next(kWideStages);
        if (++kc == C) {
          kc = 0;
          ++s;
        }
      }
      if (sr->aborted()) drain_ring(sr, pos, kWideStages);
    }
    return;
  }
  if (tid >= kWideFinish) {  // finisher
    uint32_t phase = 0;
#pragma unroll 1
    for (; left > 0; kc = 0, ++s) {
      const int chunks = min(C - kc, left);
      left -= chunks;
      if (chunks != C || left == 0) continue;  // the adders'
      if (!mbar_wait(&ctl->red_full, phase, &sr->abort)) sr->give_up(p.err);
      __syncwarp();
      lin_write<32, kWideStrip, TY>(p, red, kWideStrip, s, tid - kWideFinish);
      phase ^= 1u;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->red_empty);
    }
    return;
  }

  if (tid < kWideAdd) {  // converters
    RingPos pos, wpos;
    WideZeros cur, nxt;
    if (ZERO && left > 0) nxt.load(p.zp, p.N, groups, s * kWideStrip + row, kc / PER * 8);
#pragma unroll 1
    for (; left > 0; kc = 0, ++s) {
      const int end = kc + min(C - kc, left);
      left -= end - kc;
      const int next_row = (s + 1) * kWideStrip + row;
      if (ZERO && left > 0 && next_row < p.N) prefetch_row(p.zp + static_cast<size_t>(next_row) * groups, groups);
#pragma unroll 1
      for (int q = kc; q < end; ++q) {
        if (ZERO && (q == kc || q % PER == 0)) {
          cur = nxt;
          const int then = (q / PER + 1) * PER;
          if (then < end) nxt.load(p.zp, p.N, groups, s * kWideStrip + row, then / PER * 8);
          else if (left > 0) nxt.load(p.zp, p.N, groups, next_row, 0);
        }
        if (!mbar_wait(&sr->full[pos.at], pos.phase, &sr->abort)) sr->give_up(p.err);
        __syncwarp();
        const uint32_t codes = smem_u32(ring) + pos.at * kWideSlot + row * 128;
#pragma unroll 1
        for (int u = 0; u < UPC; ++u) {
          const uint32_t to = tmem + lanes + wpos.at * UNIT + half * (UNIT / 2);
          const uint32_t zeros = ZERO ? cur.from((q % PER) * (256 / GRP) + u * SUMS) : 0u;
          uint4 w[UNIT / 32];  // 32 codes: 16 bytes of the swizzled row
#pragma unroll
          for (int j = 0; j < UNIT / 32; ++j) w[j] = lds128(codes + (((u * (UNIT / 32) + j) ^ (row & 7)) << 4));
          // (the buffer's last unit is multiplied)
          if (!mbar_wait(&ctl->done[wpos.at], wpos.phase ^ 1u, &sr->abort)) sr->give_up(p.err);
          __syncwarp();
          tc_fence_after_sync();
#pragma unroll
          for (int j = 0; j < UNIT / 32; ++j) {
            const uint32_t zero2 = ZERO ? WideZeros::pair(zeros, j * 32 / GRP) : 0x43084308u;
            uint32_t v[16];
            w4_pairs<false>(w[j].x, zero2, reinterpret_cast<uint32_t(&)[4]>(v[0]));
            w4_pairs<false>(w[j].y, zero2, reinterpret_cast<uint32_t(&)[4]>(v[4]));
            w4_pairs<false>(w[j].z, zero2, reinterpret_cast<uint32_t(&)[4]>(v[8]));
            w4_pairs<false>(w[j].w, zero2, reinterpret_cast<uint32_t(&)[4]>(v[12]));
            tmem_st_32x32b_x16(to + j * 16, v);
          }
          tc_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->ready[wpos.at]);
          wpos.next(NA);
        }
        pos.next(kWideStages);
      }
    }
  } else {  // adders
    WideScales cur, nxt;
    if (left > 0) nxt.load(p.sc, p.N, groups, s * kWideStrip + row, kc / PER * 8);
    uint32_t red_phase = 1;
    RingPos spos;
#pragma unroll 1
    for (; left > 0; kc = 0, ++s) {
      const int end = kc + min(C - kc, left);
      left -= end - kc;
      const int next_row = (s + 1) * kWideStrip + row;
      if (left > 0 && next_row < p.N) prefetch_row(p.sc + static_cast<size_t>(next_row) * groups, groups * 2);
      float2 acc[kWideTokens / 2];
#pragma unroll
      for (int i = 0; i < kWideTokens / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll 1
      for (int q = kc; q < end; ++q) {
        if (q == kc || q % PER == 0) {
          cur = nxt;
          const int then = (q / PER + 1) * PER;
          if (then < end) nxt.load(p.sc, p.N, groups, s * kWideStrip + row, then / PER * 8);
          else if (left > 0) nxt.load(p.sc, p.N, groups, next_row, 0);
        }
#pragma unroll 1
        for (int u = 0; u < UPC; ++u) {
          const uint32_t from = tmem + lanes + kSums + spos.at * kSet + half * SUMS * 32;
          const int g = (q % PER) * (256 / GRP) + u * SUMS;
          if (!mbar_wait(&ctl->sums[spos.at], spos.phase, &sr->abort)) sr->give_up(p.err);
          __syncwarp();
          tc_fence_after_sync();
#pragma unroll
          for (int h = 0; h < SUMS; ++h) {
            const float f = cur.get(g + h);
            const float2 f2 = make_float2(f, f);
            uint32_t d[kWideTokens];
            tmem_ld_32x32b_x32(from + h * 32, d);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < kWideTokens / 2; ++i)
              acc[i] = __ffma2_rn(f2, make_float2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), acc[i]);
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->read[spos.at]);
          spos.next(ND);
        }
      }
      if (!mbar_wait(&ctl->red_empty, red_phase, &sr->abort)) sr->give_up(p.err);
#pragma unroll
      for (int i = 0; i < kWideTokens; ++i)
        if (i < p.M) red[i * kWideStrip + row] = i & 1 ? acc[i / 2].y : acc[i / 2].x;
      __syncwarp();
      if (end - kc == C && left > 0) {
        if (lane == 0) mbar_arrive(&ctl->red_full);
        red_phase ^= 1u;
      } else {  // the run's last strip, and parts of strips, whose adding up would take a warp tens of us
        bar_consumers<kWideAdders>();
        lin_finish<kWideAdders, kWideStrip, TY>(p, sp, red, kWideStrip, s, kc, end, C, b, row, &sr->last[1]);
        bar_consumers<kWideAdders>();
      }
    }
  }
  tc_fence_before_sync();
  asm volatile("bar.sync 2, %0;" ::"n"(kWideFinish + 64) : "memory");  // (and the issuers)
  if (tid < 32) tmem_dealloc(tmem, 512);
  if (sr->aborted()) drain_grace();
}

template <int GRP, bool ZERO, typename TY>
cudaError_t launch_wide(const CUtensorMap& mw, const CUtensorMap& mx, const LinParams& p, cudaStream_t s) {
  auto kern = linear_w4_wide_kernel<GRP, ZERO, TY>;
  static bool done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  const long long chunks = (static_cast<long long>(p.N) + kWideStrip - 1) / kWideStrip * (p.Kp / 256);
  int grid = device_sm_count();
  if (grid > kStreamMaxCtas) grid = kStreamMaxCtas;
  if (grid > chunks) grid = static_cast<int>(chunks);
  return launch_kernel(kern, dim3(grid), dim3(kWideBlock), kWideBytes, s, mw, mx, p);
}

template <int GRP>
cudaError_t launch_wide_types(const CUtensorMap& mw, const CUtensorMap& mx, const LinParams& p, bool f32,
                              cudaStream_t s) {
  if (p.zp) return f32 ? launch_wide<GRP, true, float>(mw, mx, p, s) : launch_wide<GRP, true, __nv_bfloat16>(mw, mx, p, s);
  return f32 ? launch_wide<GRP, false, float>(mw, mx, p, s) : launch_wide<GRP, false, __nv_bfloat16>(mw, mx, p, s);
}

}  // namespace

cudaError_t launch_linear_w4_wide(int group, const CUtensorMap& mw, const LinParams& p, bool f32, cudaStream_t s) {
  CUtensorMap mx;
  const uint64_t dims[2] = {static_cast<uint64_t>(p.Kp), static_cast<uint64_t>(p.M)};
  const uint64_t strides[1] = {static_cast<uint64_t>(p.Kp) * 2};
  const uint32_t box[2] = {64, kWideTokens};
  if (!encode_tmap(&mx, p.xp, 2, dims, strides, box)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_kernel(linear_w4_order_kernel, dim3((p.Kp + 2047) / 2048, p.M), dim3(256), 0, s, p);
  if (e != cudaSuccess) return e;
  if (group == 32) return launch_wide_types<32>(mw, mx, p, f32, s);
  if (group == 64) return launch_wide_types<64>(mw, mx, p, f32, s);
  return launch_wide_types<128>(mw, mx, p, f32, s);
}

}  // namespace moe
