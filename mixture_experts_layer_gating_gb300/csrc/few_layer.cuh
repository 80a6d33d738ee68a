// The whole MoE layer for at most 32 tokens as one cooperative launch of one
// CTA per SM (moe_layer_few).  Phases, a grid barrier between each two:
//   0  router projection into fp32 planes (slices of D); x in the k order of the
//      weight layout (perm_k), zero-padded to whole stages
//   1  CTA t: token t's planes summed, top-k softmax
//   2  every CTA lists the chosen experts and their rows; gate/up products:
//      the chosen experts' (and the shared expert's) weight stages, one equal
//      run of them per CTA, so every SM streams the same number of bytes
//      whatever the routing; a 64-column strip that two CTAs share gets one
//      partial sum from each
//   3  h = act(gate) * up of the summed strips, as a bf16 pair (hi, lo)
//   4  down products, divided up the same way
//   5  out = sum_j w_j y_j + shared, from the partial sums, one rounding
// The producer thread runs ahead of the barriers: the weights of the next
// phase are on their way while the barrier is waited for (up to 192 KB per SM).
#pragma once

#include "stream_sm103.cuh"
#include "topk_warp.cuh"

namespace moe {

constexpr int kFewMaxPlanes = 16;
constexpr int kFewMaxR = 512;  // expanded rows: 32 tokens, 16 experts each

struct FewParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* Wg;
  const float* bias;
  const void *s13, *s2, *s13s, *s2s;  // fp32 per column (e4m3) or bf16 per group (4-bit)
  __nv_bfloat16* out;
  int32_t* err;
  uint32_t* bar;  // grid barrier: arrivals at [0], generation at [16]
  float* logits;
  int32_t* ids;
  float* topw;
  float* planes;       // [nplanes][T][E]
  __nv_bfloat16* xp;   // [T][Dp]
  __nv_bfloat16* hp;   // [2][R + T][Ip] (hi, lo); row R + t: token t of the shared expert
  float* prim;         // [R + T][W]: the first partial sum of every strip of a row
  float* extra;        // [2][ctas][T][2 HC]: a CTA's part of a strip begun by an earlier one
  int T, D, E, k, I, Is, act, renorm;
  int Dp, Ip;          // padded row lengths of xp, hp (elements)
  int W;               // floats per row of prim
  int nplanes;
};

__device__ __forceinline__ float few_act(float g, float u, int act) {
  if (act == MOE_ACT_SWIGLU) return g / (1.0f + expf(-g)) * u;
  const float c = 0.7978845608028654f;  // sqrt(2 / pi)
  return 0.5f * g * (1.0f + tanhf(c * (g + 0.044715f * g * g * g))) * u;
}

template <int KIND, int GRP, int NT>
struct FewSmem {
  using Tr = StreamTraits<KIND, GRP>;
  static constexpr int kBBuf = 2 * 8 * NT * Tr::PITCH;  // hi and lo rows of one stage's k
  static constexpr int kRed = Tr::KN ? 8 * NT * (2 * Tr::HC + 4) * 4 : 0;
  static constexpr int kRedMin = 8 * NT * 68 * 4;       // the router's partial sums
  static constexpr int kRedBytes = kRed > kRedMin ? kRed : kRedMin;
  struct Ctrl {
    uint64_t full[12], empty[12];
    int abort;
    int na;
    int cnt[512];           // rows of an expert; the token's summed logits in phase 1
    uint16_t aexp[512];     // active experts, ascending
    uint16_t aoff[513];     // first sorted position of an active expert
    uint16_t amap[512];     // expert -> its index among the active
    uint16_t sid[kFewMaxR]; // expert of an expanded row
    uint16_t srow[kFewMaxR];  // expanded row at a sorted position
    uint16_t pos[kFewMaxR];   // sorted position of an expanded row
    uint16_t apos[kFewMaxR];  // active index of a sorted position
  };
  static constexpr int kOther = 3 * kBBuf + kRedBytes + static_cast<int>(sizeof(Ctrl)) + 16;
  static constexpr int NST = stream_stages(kOther);
  static constexpr int kBytes = 1024 + NST * kStageBytes + kOther;
  static_assert(NST >= 4, "too few stages");
  static_assert(kBytes <= kStreamSmemMax, "shared memory");
};

// One pass over weights: groups x strips x chunks, this CTA's run of them.
struct FewPass {
  Split sp;
  long long lo, hi;
  int S, C;  // strips of a group, chunks (stages) of a strip
};
template <int KIND, int GRP>
__device__ __forceinline__ FewPass few_pass(const FewParams& p, bool down, bool routed, int na, int G,
                                            int b) {
  using Tr = StreamTraits<KIND, GRP>;
  const int K = down ? (routed ? p.I : p.Is) : p.D;
  const int width = down ? p.D : (routed ? p.I : p.Is);
  const int per = down ? 2 * Tr::HC : Tr::HC;
  FewPass f;
  f.S = (width + per - 1) / per;
  f.C = (K + Tr::KCH - 1) / Tr::KCH;
  const int groups = routed ? na : (p.Is > 0 ? 1 : 0);
  f.sp = make_split(static_cast<long long>(groups) * f.S * f.C, G);
  f.lo = split_lo(f.sp, b);
  f.hi = split_lo(f.sp, b + 1);
  return f;
}

// Waits until all G CTAs have arrived.  Bounded: after the limit the CTA flags
// an error and goes on without waiting (every later wait ends at once).
__device__ __forceinline__ void few_grid_sync(uint32_t* bar, int G, int* abort, int32_t* err) {
  bar_consumers();
  if (threadIdx.x == 0 && !*reinterpret_cast<volatile int*>(abort)) {
    uint32_t old;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(old) : "l"(bar + 16) : "memory");
    __threadfence();
    if (atomicAdd(bar, 1u) == static_cast<uint32_t>(G - 1)) {
      *reinterpret_cast<volatile uint32_t*>(bar) = 0;
      __threadfence();
      asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(bar + 16), "r"(old + 1) : "memory");
    } else {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = 1;; ++i) {
        uint32_t now;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(bar + 16) : "memory");
        if (now != old) break;
        if ((i & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
          *reinterpret_cast<volatile int*>(abort) = 1;
          atomicOr(err, MOE_DEV_WAIT_TIMEOUT);
          break;
        }
      }
    }
    __threadfence();
  }
  bar_consumers();
}

template <int KIND, int GRP, int NT>
struct Few {
  using Tr = StreamTraits<KIND, GRP>;
  using Sm = FewSmem<KIND, GRP, NT>;
  using Ctrl = typename Sm::Ctrl;

  // ---------------------------------------------------------------- producer
  // Fills the ring with the run [f.lo, f.hi) of one pass.
  static __device__ __forceinline__ bool produce(const CUtensorMap* m, const FewPass& f, bool down,
                                                 const uint16_t* aexp, uint32_t ring, Ctrl* ctl,
                                                 uint8_t* ring_ptr, int& stage, uint32_t& phase,
                                                 uint64_t policy) {
    if (f.lo >= f.hi) return true;
    long long strip = f.lo / f.C;
    int kc = static_cast<int>(f.lo - strip * f.C);
    int a = static_cast<int>(strip / f.S), s = static_cast<int>(strip % f.S);
    for (long long q = f.lo; q < f.hi; ++q) {
      if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, &ctl->abort)) return false;
      uint64_t* bar = &ctl->full[stage];
      uint8_t* dst = ring_ptr + stage * kStageBytes;
      const int e = aexp ? aexp[a] : 0;
      mbar_arrive_expect_tx(bar, kStageBytes);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint8_t* d = dst + h * kHalfBytes;
        if (Tr::KN) {
          if (down) tma_load_3d(d, m, bar, s * 2 * Tr::HC + h * Tr::HC, kc * Tr::KCH, e, policy);
          else tma_load_4d(d, m, bar, s * Tr::HC, h, kc * Tr::KCH, e, policy);
        } else {
          if (down) tma_load_3d(d, m, bar, kc * 128, s * 128 + h * 64, e, policy);
          else tma_load_4d(d, m, bar, kc * 128, s * 64, h, e, policy);
        }
      }
      if (++stage == Sm::NST) {
        stage = 0;
        phase ^= 1u;
      }
      if (++kc == f.C) {
        kc = 0;
        if (++s == f.S) {
          s = 0;
          ++a;
        }
      }
    }
    return true;
  }

  // --------------------------------------------------------------- consumers
  // Token rows of chunk (a, kc) into buffer `buf` (cp.async, 16 bytes a piece).
  template <bool DOWN, bool ROUTED>
  static __device__ __forceinline__ void load_rows(const FewParams& p, const Ctrl* ctl, uint32_t buf,
                                                   int a, int kc, int tid) {
    constexpr int P = Tr::KCH / 8;  // pieces of a row
    constexpr int PL = DOWN ? 2 : 1;
    const int off = ROUTED ? ctl->aoff[a] : 0;
    const int n = ROUTED ? ctl->aoff[a + 1] - off : p.T;
    const int Kp = DOWN ? p.Ip : p.Dp;
    const size_t plane = static_cast<size_t>(p.T * p.k + p.T) * p.Ip;
    for (int i = tid; i < n * P * PL; i += kStreamThreads) {
      const int pc = i % P, row = (i / P) / PL, pl = (i / P) % PL;
      int src;
      if (DOWN) src = ROUTED ? off + row : p.T * p.k + row;
      else src = ROUTED ? ctl->srow[off + row] / p.k : row;
      const __nv_bfloat16* g = (DOWN ? p.hp + pl * plane : p.xp) + static_cast<size_t>(src) * Kp +
                               kc * Tr::KCH + pc * 8;
      cp_async_16(buf + pl * (8 * NT * Tr::PITCH) + row * Tr::PITCH + pc * 16, g, 16);
    }
  }

  template <bool DOWN, bool ROUTED>
  static __device__ __forceinline__ void consume(const FewParams& p, const FewPass& f, Ctrl* ctl,
                                                 uint32_t ring, uint32_t bbase, float* red, int& stage,
                                                 uint32_t& phase, int b, int G) {
    if (f.lo >= f.hi) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    constexpr uint32_t kLo = 8 * NT * Tr::PITCH;
    const int K = DOWN ? (ROUTED ? p.I : p.Is) : p.D;
    const int width = DOWN ? p.D : (ROUTED ? p.I : p.Is);
    long long strip = f.lo / f.C;
    int kc = static_cast<int>(f.lo - strip * f.C);
    int a = static_cast<int>(strip / f.S), s = static_cast<int>(strip % f.S);
    bool first_is_extra = kc != 0;  // this CTA's first strip was begun by an earlier one

    // lookahead of the token rows: two chunks
    int la = a, ls = s, lk = kc;
    long long lq = f.lo;
    auto ahead = [&](int slot) {
      if (lq < f.hi) {
        load_rows<DOWN, ROUTED>(p, ctl, bbase + slot * Sm::kBBuf, la, lk, tid);
        ++lq;
        if (++lk == f.C) {
          lk = 0;
          if (++ls == f.S) {
            ls = 0;
            ++la;
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // 4-bit weights: the group scales of the next chunk, one ahead
    W4Scales<GRP == 0 ? 128 : GRP> sc_now, sc_next;
    auto scales = [&](auto& dst, int a_, int s_, int kc_) {
      if constexpr (KIND == kStreamW4) {
        const void* base = DOWN ? (ROUTED ? p.s2 : p.s2s) : (ROUTED ? p.s13 : p.s13s);
        const int r = nk_row<KIND, GRP>(g);
        const int l0 = (DOWN ? s_ * 128 + warp * 16 : s_ * 64 + (warp & 3) * 16) + r;
        const int half = DOWN ? 0 : warp >> 2;
        const long long e = ROUTED ? ctl->aexp[a_] : 0;
        const long long row = (e * (DOWN ? 1 : 2) + half) * width + l0;
        w4_load_scales<GRP>(dst, static_cast<const __nv_bfloat16*>(base), nullptr,
                            l0 < width ? row : -1, l0 + 8 < width ? row + 8 : -1, K / GRP,
                            kc_ * (256 / GRP), lane);
      }
    };

    float acc[NT][Tr::MT][4];
    auto zero = [&]() {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < Tr::MT; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[i][j][t] = 0.0f;
    };
    zero();
    ahead(0);
    ahead(1);
    scales(sc_next, a, s, kc);
    int slot = 0, n = 0;
    for (long long q = f.lo; q < f.hi; ++q) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      bar_consumers();  // this chunk's rows are visible; the previous chunk's buffer is free
      ahead(slot == 0 ? 2 : slot - 1);
      n = ROUTED ? ctl->aoff[a + 1] - ctl->aoff[a] : p.T;
      const int ntu = (n + 7) >> 3;
      const bool strip_end = kc + 1 == f.C;
      if constexpr (KIND == kStreamW4) {
        sc_now = sc_next;
        if (q + 1 < f.hi) {
          if (!strip_end) scales(sc_next, a, s, kc + 1);
          else if (s + 1 < f.S) scales(sc_next, a, s + 1, 0);
          else scales(sc_next, a + 1, 0, 0);
        }
      }
      if (!mbar_wait(&ctl->full[stage], phase, &ctl->abort)) {
        if (lane == 0 && !*reinterpret_cast<volatile int*>(&ctl->abort)) {
          *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
          atomicOr(p.err, MOE_DEV_WAIT_TIMEOUT);
        }
      }
      __syncwarp();
      const uint32_t st = ring + stage * kStageBytes, bb = bbase + slot * Sm::kBBuf;
      if constexpr (Tr::KN) stage_mma_kn<KIND, NT, DOWN>(st, bb, kLo, warp, lane, ntu, acc);
      else if constexpr (KIND == kStreamFp8Nk)
        stage_mma_fp8nk<NT, DOWN>(st, bb, kLo, warp, lane, ntu, acc);
      else
        stage_mma_w4<GRP, NT, DOWN, false>(st, bb, kLo, warp, lane, ntu, sc_now,
                                           min(256, K - kc * 256) / GRP, acc);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->empty[stage]);
      if (++stage == Sm::NST) {
        stage = 0;
        phase ^= 1u;
      }
      slot = slot == 2 ? 0 : slot + 1;

      if (strip_end || q + 1 == f.hi) {
        // the strip's partial sum: row j, columns [0, 2 HC)
        float* dst;
        size_t pitch;
        if (first_is_extra) {
          dst = p.extra + (static_cast<size_t>(ROUTED ? 1 : 0) * kStreamMaxCtas + b) * p.T * 2 * Tr::HC;
          pitch = 2 * Tr::HC;
        } else {
          const int row0 = ROUTED ? ctl->aoff[a] : p.T * p.k;
          dst = p.prim + static_cast<size_t>(row0) * p.W + static_cast<size_t>(s) * 2 * Tr::HC;
          pitch = p.W;
        }
        first_is_extra = false;
        if constexpr (Tr::KN) {
          // four warps hold partial sums of a half's columns: added in the
          // order of k, one after another
          constexpr int RP = 2 * Tr::HC + 4;
          const int half = warp & 1, kw = warp >> 1;
#pragma unroll 1
          for (int r = 0; r < 4; ++r) {
            if (kw == r) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                if (nt < ntu) {
#pragma unroll
                  for (int mt = 0; mt < Tr::MT; ++mt) {
                    float* at = red + (nt * 8 + 2 * c) * RP + half * Tr::HC + kn_col<KIND>(lane, mt);
                    const float* v = acc[nt][mt];
                    if (r == 0) {
                      at[0] = v[0]; at[RP] = v[1]; at[1] = v[2]; at[RP + 1] = v[3];
                    } else {
                      at[0] += v[0]; at[RP] += v[1]; at[1] += v[2]; at[RP + 1] += v[3];
                    }
                  }
                }
            }
            bar_consumers();
          }
          constexpr int Q = 2 * Tr::HC / 4;
          for (int i = tid; i < n * Q; i += kStreamThreads) {
            const int row = i / Q, col = (i % Q) * 4;
            *reinterpret_cast<float4*>(dst + row * pitch + col) =
                *reinterpret_cast<const float4*>(red + row * RP + col);
          }
          bar_consumers();  // before the next strip's sums overwrite red
        } else {
          const int col = warp * 16 + nk_row<KIND, GRP>(g);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int r0 = nt * 8 + 2 * c;
            if (r0 < n) {
              dst[r0 * pitch + col] = acc[nt][0][0];
              dst[r0 * pitch + col + 8] = acc[nt][0][2];
            }
            if (r0 + 1 < n) {
              dst[(r0 + 1) * pitch + col] = acc[nt][0][1];
              dst[(r0 + 1) * pitch + col + 8] = acc[nt][0][3];
            }
          }
        }
        zero();
      }
      if (strip_end) {
        kc = 0;
        if (++s == f.S) {
          s = 0;
          ++a;
        }
      } else {
        ++kc;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    bar_consumers();
  }

  // Eight consecutive columns of one row of a strip, summed over the CTAs that
  // computed parts of it.  `at`: row r of prim, slot = the row's index inside
  // its expert, gs = the strip's index in the pass, col inside the strip.
  static __device__ __forceinline__ void gather8(const FewParams& p, const FewPass& f, bool routed,
                                                 int r, int slot, long long gs, int s, int col,
                                                 float (&v)[8]) {
    const float4* a = reinterpret_cast<const float4*>(p.prim + static_cast<size_t>(r) * p.W +
                                                      static_cast<size_t>(s) * 2 * Tr::HC + col);
    const float4 x = __ldcg(a), y = __ldcg(a + 1);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    const int c0 = split_cta(f.sp, gs * f.C), c1 = split_cta(f.sp, gs * f.C + f.C - 1);
    for (int cta = c0 + 1; cta <= c1; ++cta) {
      const float4* e = reinterpret_cast<const float4*>(
          p.extra + ((static_cast<size_t>(routed ? 1 : 0) * kStreamMaxCtas + cta) * p.T + slot) * 2 * Tr::HC +
          col);
      const float4 m = __ldcg(e), n = __ldcg(e + 1);
      v[0] += m.x; v[1] += m.y; v[2] += m.z; v[3] += m.w;
      v[4] += n.x; v[5] += n.y; v[6] += n.z; v[7] += n.w;
    }
  }
};

template <int KIND, int GRP, int NT>
__global__ void __launch_bounds__(kStreamBlock, 1)
    few_layer_kernel(const __grid_constant__ CUtensorMap m13, const __grid_constant__ CUtensorMap m2,
                     const __grid_constant__ CUtensorMap m13s, const __grid_constant__ CUtensorMap m2s,
                     const __grid_constant__ FewParams p) {
  using F = Few<KIND, GRP, NT>;
  using Tr = StreamTraits<KIND, GRP>;
  using Sm = FewSmem<KIND, GRP, NT>;
  using Ctrl = typename Sm::Ctrl;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* ring_ptr = smem_raw + pad;
  uint8_t* bptr = ring_ptr + Sm::NST * kStageBytes;
  float* red = reinterpret_cast<float*>(bptr + 3 * Sm::kBBuf);
  Ctrl* ctl = reinterpret_cast<Ctrl*>(bptr + 3 * Sm::kBBuf + Sm::kRedBytes);
  const uint32_t ring = smem_u32(ring_ptr);
  const int tid = threadIdx.x, b = blockIdx.x, G = gridDim.x;
  const int R = p.T * p.k;
  const bool shared = p.Is > 0;

  if (tid == 0) {
    for (int i = 0; i < Sm::NST; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], kStreamWarps);
    }
    ctl->abort = 0;
    fence_mbarrier_init();
  }
  __syncthreads();

  if (tid >= kStreamThreads) {  // ------------------------------------ producer
    const int lane = tid & 31;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint64_t policy = l2_policy_evict_first();
    if (lane == 0 && shared) {
      const FewPass f = few_pass<KIND, GRP>(p, false, false, 0, G, b);
      ok = F::produce(&m13s, f, false, nullptr, ring, ctl, ring_ptr, stage, phase, policy);
    }
    __syncwarp();
    asm volatile("bar.sync 2, %0;" ::"n"(kStreamBlock) : "memory");  // the expert lists are built
    if (lane == 0) {
      const int na = ctl->na;
      if (ok) ok = F::produce(&m13, few_pass<KIND, GRP>(p, false, true, na, G, b), false, ctl->aexp, ring,
                              ctl, ring_ptr, stage, phase, policy);
      if (ok && shared)
        ok = F::produce(&m2s, few_pass<KIND, GRP>(p, true, false, na, G, b), true, nullptr, ring, ctl,
                        ring_ptr, stage, phase, policy);
      if (ok) ok = F::produce(&m2, few_pass<KIND, GRP>(p, true, true, na, G, b), true, ctl->aexp, ring, ctl,
                              ring_ptr, stage, phase, policy);
      if (!ok || *reinterpret_cast<volatile int*>(&ctl->abort)) {
        // gave up: copies still in flight have to land before the CTA exits
        if (!*reinterpret_cast<volatile int*>(&ctl->abort)) {
          *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
          atomicOr(p.err, MOE_DEV_WAIT_TIMEOUT);
        }
        for (int i = 0; i < Sm::NST; ++i) {
          stage = stage == 0 ? Sm::NST - 1 : stage - 1;
          if (stage == Sm::NST - 1) phase ^= 1u;
          mbar_wait_drain(&ctl->full[stage], phase);
        }
        drain_grace();
      }
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int gtid = b * kStreamThreads + tid, gthreads = G * kStreamThreads;

  // phase 0: router planes.  A unit is 64 experts x one slice of D; its k16
  // steps go round the CTA's warps.
  {
    const int SE = (p.E + 63) / 64, steps = (p.D + 15) / 16;
    const bool vec = (p.E & 7) == 0;
    for (int u = b; u < SE * p.nplanes; u += G) {
      const int se = u % SE, pl = u / SE;
      const int s0 = static_cast<int>(static_cast<long long>(steps) * pl / p.nplanes);
      const int s1 = static_cast<int>(static_cast<long long>(steps) * (pl + 1) / p.nplanes);
      float acc[NT][4][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[i][j][t] = 0.0f;
      const int col = se * 64 + g * 8;
      for (int st = s0 + warp; st < s1; st += kStreamWarps) {
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = st * 16 + 2 * c + (i & 1) + (i >> 1) * 8;
          w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0u;
          if (k < p.D) {
            const __nv_bfloat16* src = p.Wg + static_cast<size_t>(k) * p.E + col;
            if (vec) {
              if (col < p.E) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
                w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (col + j < p.E)
                  w[i][j >> 1] |= static_cast<uint32_t>(
                                      __ldg(reinterpret_cast<const unsigned short*>(src) + j))
                                  << (16 * (j & 1));
            }
          }
        }
        uint32_t x0[NT], x1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int t = nt * 8 + g, k = st * 16 + 2 * c;
          x0[nt] = x1[nt] = 0u;
          if (t < p.T) {
            const __nv_bfloat16* src = p.x + static_cast<size_t>(t) * p.D + k;
            if (k < p.D) x0[nt] = __ldg(reinterpret_cast<const uint32_t*>(src));
            if (k + 8 < p.D) x1[nt] = __ldg(reinterpret_cast<const uint32_t*>(src + 8));
          }
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          const uint32_t a0 = __byte_perm(w[0][mt], w[1][mt], 0x5410);
          const uint32_t a1 = __byte_perm(w[0][mt], w[1][mt], 0x7632);
          const uint32_t a2 = __byte_perm(w[2][mt], w[3][mt], 0x5410);
          const uint32_t a3 = __byte_perm(w[2][mt], w[3][mt], 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_bf16(acc[nt][mt], a0, a1, a2, a3, x0[nt], x1[nt]);
        }
      }
#pragma unroll 1
      for (int r = 0; r < kStreamWarps; ++r) {
        if (warp == r) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              float* at = red + (nt * 8 + 2 * c) * 68 + g * 8 + 2 * mt;
              const float* v = acc[nt][mt];
              if (r == 0) {
                at[0] = v[0]; at[68] = v[1]; at[1] = v[2]; at[69] = v[3];
              } else {
                at[0] += v[0]; at[68] += v[1]; at[1] += v[2]; at[69] += v[3];
              }
            }
        }
        bar_consumers();
      }
      for (int i = tid; i < p.T * 64; i += kStreamThreads) {
        const int t = i >> 6, e = se * 64 + (i & 63);
        if (e < p.E) p.planes[(static_cast<size_t>(pl) * p.T + t) * p.E + e] = red[t * 68 + (i & 63)];
      }
      bar_consumers();
    }
    // x in the layout's k order, rows padded with zeros
    for (int i = gtid; i < p.T * (p.Dp / 8); i += gthreads) {
      const int t = i / (p.Dp / 8), k0 = (i % (p.Dp / 8)) * 8;
      union {
        uint4 v;
        unsigned short h[8];
      } in;
      in.v = make_uint4(0, 0, 0, 0);
      if (k0 < p.D) in.v = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * p.D + k0));
      unsigned short* dst = reinterpret_cast<unsigned short*>(p.xp) + static_cast<size_t>(t) * p.Dp;
#pragma unroll
      for (int j = 0; j < 8; ++j) dst[perm_k<KIND, GRP>(k0 + j)] = in.h[j];
    }
  }
  few_grid_sync(p.bar, G, &ctl->abort, p.err);

  // phase 1: top-k of one token per CTA
  for (int t = b; t < p.T; t += G) {
    float* sum = reinterpret_cast<float*>(ctl->cnt);
    for (int e = tid; e < p.E; e += kStreamThreads) {
      float v = 0.0f;
      for (int pl = 0; pl < p.nplanes; ++pl)
        v += __ldcg(p.planes + (static_cast<size_t>(pl) * p.T + t) * p.E + e);
      sum[e] = v;
    }
    bar_consumers();
    if (warp == 0) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = lane + 32 * i < p.E ? sum[lane + 32 * i] : 0.0f;
      warp_topk_softmax<16>(v, lane, p.E, p.k, p.renorm, p.bias, p.logits + static_cast<size_t>(t) * p.E,
                            p.ids + t * p.k, p.topw + t * p.k, p.err);
    }
    bar_consumers();
  }
  few_grid_sync(p.bar, G, &ctl->abort, p.err);

  // phase 2: the chosen experts and their rows
  for (int e = tid; e < p.E; e += kStreamThreads) ctl->cnt[e] = 0;
  for (int r = tid; r < R; r += kStreamThreads) {
    int e = __ldcg(p.ids + r);
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(p.E)) {  // only after a wait that gave up
      e = 0;
      atomicOr(p.err, MOE_DEV_BAD_EXPERT_ID);
    }
    ctl->sid[r] = static_cast<uint16_t>(e);
  }
  bar_consumers();
  for (int r = tid; r < R; r += kStreamThreads) atomicAdd(&ctl->cnt[ctl->sid[r]], 1);
  bar_consumers();
  if (warp == 0) {
    // 16 consecutive experts per lane
    int rows = 0, act = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = lane * 16 + i;
      if (e < p.E && ctl->cnt[e] > 0) {
        rows += ctl->cnt[e];
        ++act;
      }
    }
    int ir = rows, ia = act;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ur = __shfl_up_sync(0xffffffffu, ir, o), ua = __shfl_up_sync(0xffffffffu, ia, o);
      if (lane >= o) {
        ir += ur;
        ia += ua;
      }
    }
    if (lane == 31) {
      ctl->na = ia;
      ctl->aoff[ia] = static_cast<uint16_t>(ir);
    }
    int ro = ir - rows, ao = ia - act;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = lane * 16 + i;
      if (e < p.E && ctl->cnt[e] > 0) {
        ctl->aexp[ao] = static_cast<uint16_t>(e);
        ctl->aoff[ao] = static_cast<uint16_t>(ro);
        ctl->amap[e] = static_cast<uint16_t>(ao);
        ro += ctl->cnt[e];
        ++ao;
      }
    }
  }
  bar_consumers();
  for (int r = tid; r < R; r += kStreamThreads) {
    const int e = ctl->sid[r];
    int rank = 0;
    for (int q = 0; q < r; ++q) rank += ctl->sid[q] == e;
    const int a = ctl->amap[e], at = ctl->aoff[a] + rank;
    ctl->srow[at] = static_cast<uint16_t>(r);
    ctl->apos[at] = static_cast<uint16_t>(a);
    ctl->pos[r] = static_cast<uint16_t>(at);
  }
  __threadfence_block();
  asm volatile("bar.arrive 2, %0;" ::"n"(kStreamBlock) : "memory");
  bar_consumers();
  const int na = ctl->na;

  int stage = 0;
  uint32_t phase = 0;
  const uint32_t bbase = smem_u32(bptr);
  const FewPass us = few_pass<KIND, GRP>(p, false, false, na, G, b);
  const FewPass ur = few_pass<KIND, GRP>(p, false, true, na, G, b);
  if (shared) F::template consume<false, false>(p, us, ctl, ring, bbase, red, stage, phase, b, G);
  F::template consume<false, true>(p, ur, ctl, ring, bbase, red, stage, phase, b, G);
  few_grid_sync(p.bar, G, &ctl->abort, p.err);

  // phase 3: h = act(gate) * up, as a bf16 pair in the k order of the down pass
  {
    const int per = p.Ip / 8;
    const int rows = R + (shared ? p.T : 0);
    const size_t plane = static_cast<size_t>(R + p.T) * p.Ip;
    for (int i = gtid; i < rows * per; i += gthreads) {
      const int r = i / per, k0 = (i % per) * 8;
      const bool rt = r < R;
      const int width = rt ? p.I : p.Is;
      float h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = 0.0f;
      if (k0 < width) {
        const FewPass& f = rt ? ur : us;
        const int a = rt ? ctl->apos[r] : 0;
        const int sl = rt ? r - ctl->aoff[a] : r - R;
        const int s = k0 / Tr::HC, col = k0 % Tr::HC;
        const long long gs = static_cast<long long>(a) * f.S + s;
        float u[8];
        F::gather8(p, f, rt, r, sl, gs, s, col, h);
        F::gather8(p, f, rt, r, sl, gs, s, col + Tr::HC, u);
        if constexpr (KIND == kStreamFp8 || KIND == kStreamFp8Nk) {
          const float* sc = static_cast<const float*>(rt ? p.s13 : p.s13s) +
                            (rt ? static_cast<size_t>(ctl->aexp[a]) * 2 * width : 0);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h[j] *= __ldg(sc + k0 + j);
            u[j] *= __ldg(sc + width + k0 + j);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = few_act(h[j], u[j], p.act);
      }
      __nv_bfloat16* dst = p.hp + static_cast<size_t>(r) * p.Ip;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        __nv_bfloat16 hi, lo;
        split_bf16(h[j], hi, lo);
        const int at = perm_k<KIND, GRP>(k0 + j);
        dst[at] = hi;
        dst[plane + at] = lo;
      }
    }
  }
  few_grid_sync(p.bar, G, &ctl->abort, p.err);

  // phase 4: down products
  const FewPass ds = few_pass<KIND, GRP>(p, true, false, na, G, b);
  const FewPass dr = few_pass<KIND, GRP>(p, true, true, na, G, b);
  if (shared) F::template consume<true, false>(p, ds, ctl, ring, bbase, red, stage, phase, b, G);
  F::template consume<true, true>(p, dr, ctl, ring, bbase, red, stage, phase, b, G);
  few_grid_sync(p.bar, G, &ctl->abort, p.err);

  // phase 5: the weighted sum of a token's rows, j ascending, the shared row last
  {
    const int per = p.D / 8;
    for (int i = gtid; i < p.T * per; i += gthreads) {
      const int t = i / per, d0 = (i % per) * 8;
      const int s = d0 / (2 * Tr::HC), col = d0 % (2 * Tr::HC);
      float o[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = 0.0f;
      for (int j = 0; j < p.k; ++j) {
        const int r = ctl->pos[t * p.k + j], a = ctl->apos[r];
        F::gather8(p, dr, true, r, r - ctl->aoff[a], static_cast<long long>(a) * dr.S + s, s, col, y);
        if constexpr (KIND == kStreamFp8 || KIND == kStreamFp8Nk) {
          const float* sc = static_cast<const float*>(p.s2) + static_cast<size_t>(ctl->aexp[a]) * p.D + d0;
#pragma unroll
          for (int q = 0; q < 8; ++q) y[q] *= __ldg(sc + q);
        }
        const float w = __ldcg(p.topw + t * p.k + j);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = fmaf(w, y[q], o[q]);
      }
      if (shared) {
        F::gather8(p, ds, false, R + t, t, s, s, col, y);
        if constexpr (KIND == kStreamFp8 || KIND == kStreamFp8Nk) {
          const float* sc = static_cast<const float*>(p.s2s) + d0;
#pragma unroll
          for (int q = 0; q < 8; ++q) y[q] *= __ldg(sc + q);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] += y[q];
      }
      union {
        uint4 v;
        __nv_bfloat16 h[8];
      } w;
#pragma unroll
      for (int q = 0; q < 8; ++q) w.h[q] = __float2bfloat16_rn(o[q]);
      *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(t) * p.D + d0) = w.v;
    }
  }
}

// ------------------------------------------------------------------ launch
struct FewArgs {
  FewParams p;
  const void *W13, *W2, *W13s, *W2s;
};

// The tensor maps of one expert projection pair.  G = experts (1: shared).
template <int KIND, int GRP>
bool few_maps(const void* W13, const void* W2, int G, int D, int I, CUtensorMap& m13, CUtensorMap& m2) {
  using Tr = StreamTraits<KIND, GRP>;
  const uint64_t g = G, d = D, n = I;
  if (Tr::KN) {
    const uint64_t eb = KIND == kStreamBf16 ? 2 : 1;
    const auto dt = KIND == kStreamBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const uint64_t d13[4] = {n, 2, d, g}, t13[3] = {n * eb, 2 * n * eb, d * 2 * n * eb};
    const uint32_t b13[4] = {Tr::HC, 1, 64, 1};
    const uint64_t d2[3] = {d, n, g}, t2[2] = {d * eb, n * d * eb};
    const uint32_t b2[3] = {Tr::HC, 64, 1};
    return encode_tmap(&m13, W13, 4, d13, t13, b13, dt) && encode_tmap(&m2, W2, 3, d2, t2, b2, dt);
  }
  const uint64_t kb = KIND == kStreamFp8Nk ? d : d / 2, nb = KIND == kStreamFp8Nk ? n : n / 2;
  const uint64_t d13[4] = {kb, n, 2, g}, t13[3] = {kb, n * kb, 2 * n * kb};
  const uint32_t b13[4] = {128, 64, 1, 1};
  const uint64_t d2[3] = {nb, d, g}, t2[2] = {nb, d * nb};
  const uint32_t b2[3] = {128, 64, 1};
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return encode_tmap(&m13, W13, 4, d13, t13, b13, u8) && encode_tmap(&m2, W2, 3, d2, t2, b2, u8);
}

template <int KIND, int GRP, int NT>
cudaError_t launch_few_nt(const FewArgs& a, cudaStream_t s) {
  using Sm = FewSmem<KIND, GRP, NT>;
  auto kern = few_layer_kernel<KIND, GRP, NT>;
  static bool done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  CUtensorMap m13, m2, m13s, m2s;
  if (!few_maps<KIND, GRP>(a.W13, a.W2, a.p.E, a.p.D, a.p.I, m13, m2)) return cudaErrorInvalidValue;
  if (a.p.Is > 0) {
    if (!few_maps<KIND, GRP>(a.W13s, a.W2s, 1, a.p.D, a.p.Is, m13s, m2s)) return cudaErrorInvalidValue;
  } else {
    m13s = m13;
    m2s = m2;
  }
  int sms = device_sm_count();
  if (sms > kStreamMaxCtas) sms = kStreamMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(kStreamBlock);
  cfg.dynamicSmemBytes = Sm::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // all CTAs resident: they wait for one another
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, m13, m2, m13s, m2s, a.p);
}

template <int KIND, int GRP>
cudaError_t launch_few_kind(const FewArgs& a, cudaStream_t s) {
  if (a.p.T <= 8) return launch_few_nt<KIND, GRP, 1>(a, s);
  if (a.p.T <= 16) return launch_few_nt<KIND, GRP, 2>(a, s);
  return launch_few_nt<KIND, GRP, 4>(a, s);
}

cudaError_t launch_few_bf16(const FewArgs& a, cudaStream_t s);
cudaError_t launch_few_fp8(const FewArgs& a, cudaStream_t s);
cudaError_t launch_few_fp8nk(const FewArgs& a, cudaStream_t s);
cudaError_t launch_few_w4(int group, const FewArgs& a, cudaStream_t s);

}  // namespace moe
