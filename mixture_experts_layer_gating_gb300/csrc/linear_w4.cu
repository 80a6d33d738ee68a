// y = x W^T for a few rows of x and 4-bit weights with group scales (moe_linear_w4;
// linear_w4_wide.cu has it for more), and the weights' way into and out of the 4-bit form.
//
//   y[m][n] = sum over groups q of s[n][q] * (sum over the group's k of
//             (code[n][k] - zero[n][q]) * x[m][k])
//
// The codes are made bf16 in the registers that mma.sync reads, a group's sum (fp32,
// its first product starts from zero) is multiplied by the group's scale and added
// in fp32.  Strips of 128 output features x stages of 256 k are divided into equal
// runs over the CTAs, so that every SM streams as many bytes whatever N; the parts
// of a strip that several CTAs share are added by the one that arrives last.
//
// In a graph, weights from HBM: 8192 x 8192, groups of 128, one row 15.0 us (35 MB; HBM
// floor 5.2; with zero points 16.5), four 17.3, eight 17.5, sixteen 20.0; 2048 x 2048, one
// row 6.1 (a call from Python after another: 6.6, of which the host takes 5.8); 13 rows x
// 2816 x 4224, groups of 32, 12.8.  What bounds it: a CTA has 13 stages
// at 8192 x 8192, each 645 cycles of conversions and products (HBM brings one in 697),
// after the launch and the first bytes (4 us) and before the shared strips' sums (3).
#include "linear_w4.cuh"

namespace moe {

namespace {

template <int GRP, int NT>
struct LinSmem {
  using Tr = StreamTraits<kStreamW4, GRP>;
  static constexpr int kTeams = 2;
  static constexpr int kCons = 32 * kStreamWarps * kTeams;
  static constexpr int kFeeders = 2;  // feeder warps
  static constexpr int kBlock = kCons + 32 + 32 * kFeeders + 32;  // + producer, feeders, finisher
  static constexpr int kSlot = stream_slot(8 * NT * Tr::PITCH);
  static constexpr int kRP = 128 + 4;
  static constexpr int kRedBytes = 8 * NT * kRP * 4;
  static constexpr int kRedBufs = 2;
  static constexpr int kOther = kRedBufs * kRedBytes + static_cast<int>(sizeof(StreamRing)) + 16;
  static constexpr int NST = stream_stages(kSlot, kOther);
  static constexpr int kBytes = 1024 + NST * kSlot + kOther;
  static_assert(NST >= 4 && NST % kFeeders == 0 && kBytes <= kStreamSmemMax, "shared memory");
};

// Who finishes a strip: all consumers the run's last one, when they have nothing
// else to do, shared ones of more than two rows and any of more than eight (one
// warp takes about 0.4 us a row, 16 rows longer than a short strip streams); the
// finisher warp the others.
__device__ __forceinline__ bool lin_by_consumers(int M, int C, int chunks, int left) {
  return left == 0 || M > 8 || (M > 2 && chunks != C);
}

// Strips of 128 output features x stages of 256 k, divided into equal runs over
// the CTAs.
template <int GRP, int NT, bool ZERO, typename TY>
__global__ void __launch_bounds__(LinSmem<GRP, NT>::kBlock, 1)
    linear_w4_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ LinParams p) {
  using Tr = StreamTraits<kStreamW4, GRP>;
  using Sm = LinSmem<GRP, NT>;
  constexpr int CT = Sm::kCons, RP = Sm::kRP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* red = reinterpret_cast<float*>(ring + Sm::NST * Sm::kSlot);
  StreamRing* sr = reinterpret_cast<StreamRing*>(ring + Sm::NST * Sm::kSlot + Sm::kRedBufs * Sm::kRedBytes);
  const int tid = threadIdx.x, b = blockIdx.x, lane = tid & 31;
  const int C = (p.K + 255) / 256, S = (p.N + kLinStrip - 1) / kLinStrip;
  const Split sp = make_split(static_cast<long long>(S) * C, gridDim.x);
  const long long lo = split_lo(sp, b), hi = split_lo(sp, b + 1);

  if (tid == 0) sr->init(CT / 32);
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  int s = static_cast<int>(lo / C), kc = static_cast<int>(lo % C);

  if (tid >= CT + 32 + 32 * Sm::kFeeders) {  // finisher: the strips that the consumers leave to it
    RingPos rpos;
    int left = static_cast<int>(hi - lo);
#pragma unroll 1
    for (; left > 0; kc = 0, ++s) {
      const int chunks = min(C - kc, left);
      left -= chunks;
      if (lin_by_consumers(p.M, C, chunks, left)) continue;
      if (!mbar_wait(&sr->red_full[rpos.at], rpos.phase, &sr->abort)) sr->give_up(p.err);
      __syncwarp();
      lin_finish<32, kLinStrip, TY>(p, sp, red + rpos.at * (Sm::kRedBytes / 4), RP, s, kc, kc + chunks, C, b, lane, &sr->last[0]);
      __syncwarp();
      mbar_arrive(&sr->red_empty[rpos.at]);
      rpos.next(Sm::kRedBufs);
    }
    return;
  }
  if (tid >= CT + 32) {  // feeders: x rows of every kFeeders-th stage, always the same slots: a
    // wait cannot mistake a fill for the one before
    int left = static_cast<int>(hi - lo);
    const int first = (tid - CT - 32) >> 5;  // of the run's stages
    RingPos pos;
    pos.skip(first, Sm::NST);
    kc = (kc + first) % C;
    left -= first;
    // 32 pieces of 8 inputs a row, one a lane, put in order on the way; the next stage's are loaded before this one's slot is waited for
    const uint32_t pdst = perm_k<kStreamW4, GRP>(lane * 8) * 2;
    uint4 x[8 * NT];
    auto load = [&](int kc_) {
      const int k0 = kc_ * 256 + lane * 8;
#pragma unroll
      for (int i = 0; i < 8 * NT; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (i < p.M && k0 < p.K) x[i] = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(i) * p.K + k0));
      }
    };
    if (left > 0) load(kc);
#pragma unroll 1
    for (; left > 0; left -= Sm::kFeeders) {
      if (!mbar_wait(&sr->empty[pos.at], pos.phase ^ 1u, &sr->abort)) {
        sr->give_up(p.err);
        break;
      }
      uint8_t* dst = ring + pos.at * Sm::kSlot + kStageBytes + pdst;
#pragma unroll
      for (int i = 0; i < 8 * NT; ++i) {
        if (i >= p.M) break;
        uint4 v;
        v.x = __byte_perm(x[i].x, x[i].z, 0x5410);
        v.y = __byte_perm(x[i].x, x[i].z, 0x7632);
        v.z = __byte_perm(x[i].y, x[i].w, 0x5410);
        v.w = __byte_perm(x[i].y, x[i].w, 0x7632);
        *reinterpret_cast<uint4*>(dst + i * Tr::PITCH) = v;
      }
      mbar_arrive(&sr->full[pos.at]);
      pos.skip(Sm::kFeeders, Sm::NST);
      kc = (kc + Sm::kFeeders) % C;
      if (left > Sm::kFeeders) load(kc);
    }
    return;
  }
  if (tid >= CT) {  // producer
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_first();
      RingPos pos;
      for (long long q = lo; q < hi; ++q) {
        if (!mbar_wait(&sr->empty[pos.at], pos.phase ^ 1u, &sr->abort)) {
          sr->give_up(p.err);
          break;
        }
        mbar_arrive_expect_tx(&sr->full[pos.at], kStageBytes);
        tma_load_2d(ring + pos.at * Sm::kSlot, &mw, &sr->full[pos.at], kc * 128, s * kLinStrip, policy);
        pos.next(Sm::NST);
        if (++kc == C) {
          kc = 0;
          ++s;
        }
      }
      if (sr->aborted()) drain_ring(sr, pos, Sm::NST);
    }
    return;
  }

  // consumers
  const int team = Sm::kTeams == 1 ? 0 : tid / (32 * kStreamWarps);
  const int warp = (tid >> 5) % kStreamWarps, g = lane >> 2, c = lane & 3;
  const uint32_t ring_a = smem_u32(ring);
  const int r = nk_row<kStreamW4, GRP>(g), groups = p.K / GRP;
  const int ntu = (p.M + 7) >> 3;
  RingPos ring_pos, rpos;
  // the lane's row of group scales, loaded two of the team's chunks ahead, a strip's
  // first ones while the strip before it is summed up
  const int qh = (warp & 1) * (128 / GRP);
  W4Scales<GRP, ZERO> sc0, sc1;
  long long srow = -1;
  auto first_scales = [&](int s_, int kc_) {
    const int n = s_ * kLinStrip + (warp >> 1) * 32 + (c >> 1) * 16 + r + (c & 1) * 8;
    srow = n < p.N ? static_cast<long long>(n) * groups : -1;
    w4_load_scales<GRP, ZERO>(sc0, p.sc, p.zp, srow, groups, (kc_ + team) * (256 / GRP) + qh);
    w4_load_scales<GRP, ZERO>(sc1, p.sc, p.zp, srow, groups, (kc_ + team + Sm::kTeams) * (256 / GRP) + qh);
  };
  if (lo < hi) first_scales(s, kc);
  float acc[NT][2][4];
#pragma unroll 1
  for (int left = static_cast<int>(hi - lo); left > 0; kc = 0, ++s) {  // a strip, or this CTA's part of it
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][j][t] = 0.0f;
    const int chunks = min(C - kc, left), end = kc + chunks;
    RingPos pos = ring_pos;
    if (team) pos.next(Sm::NST);
    auto step = [&](W4Scales<GRP, ZERO>& sc, int q) {
      if (!mbar_wait(&sr->full[pos.at], pos.phase, &sr->abort)) sr->give_up(p.err);
      __syncwarp();
      const uint32_t st = ring_a + pos.at * Sm::kSlot;
      stage_mma_w4<GRP, NT, NT, NT == 2 ? 1 : 2, ZERO, false>(st, st + kStageBytes, warp, lane, ntu, sc, acc);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sr->empty[pos.at]);
      pos.skip(Sm::kTeams, Sm::NST);
      w4_load_scales<GRP, ZERO>(sc, p.sc, p.zp, srow, groups, (q + 2 * Sm::kTeams) * (256 / GRP) + qh);
    };
    // two by two, each with scales of its own: moving them on from one step to the
    // next would wait for the loads
#pragma unroll 1
    for (int q = kc + team; q < end; q += Sm::kTeams) {
      step(sc0, q);
      if ((q += Sm::kTeams) >= end) break;
      step(sc1, q);
    }
    ring_pos.skip(chunks % Sm::NST, Sm::NST);
    ring_pos.phase ^= (chunks / Sm::NST) & 1;
    left -= chunks;
    if (left > 0) first_scales(s + 1, 0);
    add_sums<kStreamW4, GRP, NT, Sm::kTeams, RP>(red + rpos.at * (Sm::kRedBytes / 4), team, warp, lane, ntu, acc, [&]() {
      if (!mbar_wait(&sr->red_empty[rpos.at], rpos.phase ^ 1u, &sr->abort)) sr->give_up(p.err);
      __syncwarp();
    }, [] { bar_consumers<CT>(); });
    if (lin_by_consumers(p.M, C, chunks, left)) {
      bar_consumers<CT>();
      lin_finish<CT, kLinStrip, TY>(p, sp, red + rpos.at * (Sm::kRedBytes / 4), RP, s, kc, end, C, b, tid, &sr->last[1]);
      bar_consumers<CT>();
    } else {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sr->red_full[rpos.at]);
      rpos.next(Sm::kRedBufs);
    }
  }
  if (sr->aborted()) drain_grace();
}

template <int GRP, int NT, bool ZERO, typename TY>
cudaError_t launch_lin(const CUtensorMap& m, const LinParams& p, int grid, cudaStream_t s) {
  using Sm = LinSmem<GRP, NT>;
  auto kern = linear_w4_kernel<GRP, NT, ZERO, TY>;
  static bool done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  return launch_kernel(kern, dim3(grid), dim3(Sm::kBlock), Sm::kBytes, s, m, p);
}

template <int GRP, int NT>
cudaError_t launch_lin_types(const CUtensorMap& m, const LinParams& p, bool f32, int grid, cudaStream_t s) {
  if (p.zp)
    return f32 ? launch_lin<GRP, NT, true, float>(m, p, grid, s)
               : launch_lin<GRP, NT, true, __nv_bfloat16>(m, p, grid, s);
  return f32 ? launch_lin<GRP, NT, false, float>(m, p, grid, s)
             : launch_lin<GRP, NT, false, __nv_bfloat16>(m, p, grid, s);
}

template <int GRP>
cudaError_t launch_lin_rows(const CUtensorMap& m, const LinParams& p, bool f32, int grid, cudaStream_t s) {
  if (p.M <= 8) return launch_lin_types<GRP, 1>(m, p, f32, grid, s);
  return launch_lin_types<GRP, 2>(m, p, f32, grid, s);
}

// ------------------------------------------------------------ 4-bit weights
constexpr int kQCols = 64;

// One group of 64 columns per block, four threads a column: its largest |w|, scale =
// bf16(amax / 7), codes round(w / scale) + 8 in [0, 15].  8 x 4096 x 4096, groups of
// 64: 177 us from bf16 (1.9 TB/s), 171 from fp32 (3.6 TB/s); what bounds it is the
// division of every weight by its scale.  It runs once, when weights are loaded.
template <int GRP, typename T>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const T* __restrict__ W, int K, int N,
                                                          uint8_t* __restrict__ q,
                                                          __nv_bfloat16* __restrict__ sc) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float tile[GRP][kQCols + 1];
  __shared__ uint32_t most[4][kQCols];
  __shared__ float scale[kQCols];
  const int tid = threadIdx.x, n0 = blockIdx.x * kQCols, kg = blockIdx.y;
  const size_t mat = blockIdx.z;
  const T* src = W + mat * K * N + static_cast<size_t>(kg) * GRP * N;
  const int col = tid % kQCols, part = tid / kQCols;
  float v[GRP / 4];
#pragma unroll
  for (int i = 0; i < GRP / 4; ++i)
    v[i] = n0 + col < N ? static_cast<float>(src[static_cast<size_t>(part + 4 * i) * N + n0 + col]) : 0.0f;
  uint32_t m = 0;  // bits of non-negative floats order as the floats do, infinity and NaN highest
#pragma unroll
  for (int i = 0; i < GRP / 4; ++i) {
    m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    tile[part + 4 * i][col] = v[i];
  }
  most[part][col] = m;
  __syncthreads();
  if (tid < kQCols) {
    m = max(max(most[0][tid], most[1][tid]), max(most[2][tid], most[3][tid]));
    float s = __bfloat162float(__float2bfloat16_rn(__uint_as_float(m) / 7.0f));
    if (m >= 0x7f800000u) s = __int_as_float(0x7fc00000);  // a group with an Inf or NaN: its products are NaN
    else if (s == 0.0f) s = 1.0f;                          // all zeros (or below the scale's range)
    scale[tid] = s;
    if (n0 + tid < N) sc[(mat * N + n0 + tid) * (K / GRP) + kg] = __float2bfloat16_rn(s);
  }
  __syncthreads();
  constexpr int WORDS = GRP / 8;
  for (int i = tid; i < kQCols * WORDS; i += 256) {
    const int n = i / WORDS, w = i % WORDS;
    if (n0 + n >= N) continue;
    const float s = scale[n];
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = rintf(tile[8 * w + j][n] / s);
      const int u = isnan(t) ? 8 : static_cast<int>(fminf(fmaxf(t, -8.0f), 7.0f)) + 8;
      v |= static_cast<uint32_t>(u) << (4 * j);
    }
    *reinterpret_cast<uint32_t*>(q + (mat * N + n0 + n) * (K / 2) + static_cast<size_t>(kg) * (GRP / 2) + 4 * w) = v;
  }
}

// W[k][n] = bf16((code - zero) * scale), back in the [.., K, N] layout.  A group of 64
// columns per block, turned round in shared memory.  8 x 4096 x 4096, groups of 64: 99
// us (3.5 TB/s; floor 51).
template <int GRP>
__global__ void __launch_bounds__(256) dequantize_w4_kernel(const uint8_t* __restrict__ q,
                                                            const __nv_bfloat16* __restrict__ sc,
                                                            const uint8_t* __restrict__ zp, int K, int N,
                                                            __nv_bfloat16* __restrict__ W) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ __nv_bfloat16 tile[GRP][kQCols + 2];
  const int tid = threadIdx.x, n0 = blockIdx.x * kQCols, kg = blockIdx.y;
  const size_t mat = blockIdx.z;
  constexpr int WORDS = GRP / 8;
  for (int i = tid; i < kQCols * WORDS; i += 256) {
    const int n = i / WORDS, w = i % WORDS;
    if (n0 + n >= N) continue;
    const size_t row = mat * N + n0 + n;
    const uint32_t v =
        *reinterpret_cast<const uint32_t*>(q + row * (K / 2) + static_cast<size_t>(kg) * (GRP / 2) + 4 * w);
    const size_t at = row * (K / GRP) + kg;
    const float s = __bfloat162float(sc[at]);
    const int z = zp ? zp[at] & 15 : 8;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[8 * w + j][n] = __float2bfloat16_rn(static_cast<float>(static_cast<int>((v >> (4 * j)) & 15u) - z) * s);
  }
  __syncthreads();
  __nv_bfloat16* dst = W + mat * K * N + static_cast<size_t>(kg) * GRP * N;
  for (int i = tid; i < GRP * kQCols; i += 256) {
    const int k = i / kQCols, n = i % kQCols;
    if (n0 + n < N) dst[static_cast<size_t>(k) * N + n0 + n] = tile[k][n];
  }
}

template <int GRP>
cudaError_t launch_quantize(const void* W, bool f32, long long G, int K, int N, uint8_t* q,
                            __nv_bfloat16* sc, cudaStream_t s) {
  const dim3 grid((N + kQCols - 1) / kQCols, K / GRP, static_cast<unsigned>(G));
  if (f32)
    return launch_kernel(quantize_w4_kernel<GRP, float>, grid, dim3(256), 0, s, static_cast<const float*>(W),
                         K, N, q, sc);
  return launch_kernel(quantize_w4_kernel<GRP, __nv_bfloat16>, grid, dim3(256), 0, s,
                       static_cast<const __nv_bfloat16*>(W), K, N, q, sc);
}

template <int GRP>
cudaError_t launch_dequantize(const uint8_t* q, const __nv_bfloat16* sc, const uint8_t* zp, long long G,
                              int K, int N, __nv_bfloat16* W, cudaStream_t s) {
  const dim3 grid((N + kQCols - 1) / kQCols, K / GRP, static_cast<unsigned>(G));
  return launch_kernel(dequantize_w4_kernel<GRP>, grid, dim3(256), 0, s, q, sc, zp, K, N, W);
}

}  // namespace

// A product's scratch: arrival counts, partial sums, ordered rows.
LinearW4Scratch linear_w4_scratch(int M, int K, int N) {
  const bool wide = linear_w4_wide(M, K, N);
  const size_t Kp = (static_cast<size_t>(K) + 255) / 256 * 256;
  LinearW4Scratch l{};
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur = (cur + bytes + 255) / 256 * 256;
    return o;
  };
  l.cnt = take(kStreamMaxCtas * 4);
  l.part = take(static_cast<size_t>(kStreamMaxCtas) * 2 * M * (wide ? kWideStrip : kLinStrip) * 4);
  l.xp = take(wide ? static_cast<size_t>(M) * Kp * 2 : 0);
  l.total = cur;
  return l;
}

cudaError_t launch_linear_w4(int M, int K, int N, int group, const void* x, const void* wq, const void* sc,
                             const uint8_t* zp, void* y, bool y_f32, int32_t* err, uint8_t* scratch, cudaStream_t s) {
  CUtensorMap m;
  const uint64_t dims[2] = {static_cast<uint64_t>(K) / 2, static_cast<uint64_t>(N)};
  const uint64_t strides[1] = {static_cast<uint64_t>(K) / 2};
  const bool wide = linear_w4_wide(M, K, N);
  const uint32_t box[2] = {128, static_cast<uint32_t>(wide ? kWideStrip : kLinStrip)};
  if (!encode_tmap(&m, wq, 2, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8)) return cudaErrorInvalidValue;
  LinParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.sc = static_cast<const __nv_bfloat16*>(sc);
  p.zp = zp;
  p.y = y;
  p.err = err;
  const LinearW4Scratch l = linear_w4_scratch(M, K, N);
  p.cnt = reinterpret_cast<int32_t*>(scratch + l.cnt);
  p.part = reinterpret_cast<float*>(scratch + l.part);
  p.xp = reinterpret_cast<__nv_bfloat16*>(scratch + l.xp);
  p.M = M;
  p.K = K;
  p.N = N;
  p.Kp = (K + 255) / 256 * 256;
  if (wide) return launch_linear_w4_wide(group, m, p, y_f32, s);
  const long long chunks = (static_cast<long long>(N) + kLinStrip - 1) / kLinStrip * ((K + 255) / 256);
  int grid = device_sm_count();
  if (grid > kStreamMaxCtas) grid = kStreamMaxCtas;
  if (grid > chunks) grid = static_cast<int>(chunks);
  if (group == 32) return launch_lin_rows<32>(m, p, y_f32, grid, s);
  if (group == 64) return launch_lin_rows<64>(m, p, y_f32, grid, s);
  return launch_lin_rows<128>(m, p, y_f32, grid, s);
}

cudaError_t launch_quantize_w4(const void* W, bool f32, long long G, int K, int N, int group, void* q,
                               void* sc, cudaStream_t s) {
  auto* qq = static_cast<uint8_t*>(q);
  auto* ss = static_cast<__nv_bfloat16*>(sc);
  if (group == 32) return launch_quantize<32>(W, f32, G, K, N, qq, ss, s);
  if (group == 64) return launch_quantize<64>(W, f32, G, K, N, qq, ss, s);
  return launch_quantize<128>(W, f32, G, K, N, qq, ss, s);
}

cudaError_t launch_dequantize_w4(const void* q, const void* sc, const uint8_t* zp, long long G, int K, int N,
                                 int group, void* W, cudaStream_t s) {
  auto* qq = static_cast<const uint8_t*>(q);
  auto* ss = static_cast<const __nv_bfloat16*>(sc);
  auto* ww = static_cast<__nv_bfloat16*>(W);
  if (group == 32) return launch_dequantize<32>(qq, ss, zp, G, K, N, ww, s);
  if (group == 64) return launch_dequantize<64>(qq, ss, zp, G, K, N, ww, s);
  return launch_dequantize<128>(qq, ss, zp, G, K, N, ww, s);
}

}  // namespace moe
