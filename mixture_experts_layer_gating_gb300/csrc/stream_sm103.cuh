// Building blocks of the kernels for a few tokens (few_layer.cuh,
// linear_w4.cu): weights streamed once from HBM through a ring of 16 KB
// shared-memory stages that one thread fills with TMA box loads, multiplied by
// at most 32 token rows with mma.sync (m16n8k16, the weights as the 16-row
// operand and the tokens as the 8 columns).
//
// Why mma.sync and not tcgen05: at a few tokens every weight is used for a
// handful of multiply-adds, so the tensor rate is no limit (one SM's share of
// HBM, ~24 bytes a cycle, feeds one m16n8k16 every 20 to 40 cycles), while a
// tcgen05 operand has to lie in shared memory in its final type: 8- and 4-bit
// weights would be expanded to bf16 there, written and read once more.  With
// mma.sync they are expanded in the registers that the multiply reads.
//
// Roles of a CTA: consumer warps in one or two teams of eight (two teams take
// the stages in turn and add their sums at the end of a strip: twice the time
// per stage for the latencies of a stage's loads, conversions and multiplies),
// a producer warp (weights) and feeder warps (the token rows of a stage, put
// beside its weights; the feeders take the stages in turn).
//
// Operand types: bf16 weights are multiplied as bf16; e4m3 weights and 4-bit
// codes (exact there) as fp16, by token rows that are fp16 times a power of
// two that puts the row's largest element in [2^14, 2^15).  One conversion
// makes two e4m3 values fp16, and an fp16 row needs no second term for h.
//
// A stage is two boxes ("halves") of 64 rows x 128 bytes, 128-byte swizzled:
//   [.., K, N] weights (bf16, e4m3): 64 consecutive k, 64 or 128 columns a half;
//     warp w multiplies k 16 (w / 2) .. + 15 of half w % 2, so the four warps of
//     a half hold partial sums of the same columns;
//   [.., N, K] weights (e4m3, 4-bit): 64 output rows a half, 128 or 256
//     consecutive k; warp w owns rows 16 w .. + 15 of the 128 and all the k.
// The k order inside an mma is free as long as both operands use the same:
// each layout takes the order in which a thread's 16-byte shared loads hold its
// operand registers, and the token rows are stored in that order (perm_k).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "moe_internal.h"
#include "sm103_ptx.cuh"

namespace moe {

constexpr int kStageBytes = 16384;
constexpr int kHalfBytes = 8192;
constexpr int kStreamWarps = 8;     // consumer warps of a team
constexpr int kStreamMaxCtas = 160; // most CTAs of a launch
constexpr int kStreamMaxRows = 32;  // most token rows
constexpr int kMaxStages = 12;      // of the ring

enum StreamKind : int { kStreamBf16 = 0, kStreamFp8 = 1, kStreamFp8Nk = 2, kStreamW4 = 3 };

template <int KIND, int GRP>
struct StreamTraits {
  static constexpr bool KN = KIND == kStreamBf16 || KIND == kStreamFp8;
  static constexpr int KCH = KN ? 64 : (KIND == kStreamFp8Nk ? 128 : 256);  // k of a stage
  static constexpr int HC = KIND == kStreamFp8 ? 128 : 64;  // output columns of a half
  static constexpr int MT = KN ? HC / 16 : 1;               // 16-column mma tiles of a warp
  // bytes between token rows in shared memory: the padding makes a quarter-
  // (KN: half-) warp's loads of several rows fall on different banks
  static constexpr int PITCH = KCH * 2 + (KN ? 32 : 64);
  static constexpr bool F16 = KIND != kStreamBf16;  // operand type of moe_layer_few
};

// Position of input k in a token row as the kernels store it (a bijection
// inside every block of 16, 64 or GRP inputs).
template <int KIND, int GRP>
__host__ __device__ __forceinline__ int perm_k(int k) {
  if (KIND == kStreamBf16 || KIND == kStreamFp8)
    return (k & ~15) | ((k & 6) << 1) | ((k & 8) >> 2) | (k & 1);
  if (KIND == kStreamFp8Nk) return (k & ~63) | ((k & 8) << 2) | ((k & 48) >> 1) | (k & 7);
  constexpr int Q = GRP ? GRP : 32, J = Q / 32;  // J: 8-k words of a thread in a group
  const int q = k / Q, r = k % Q;
  const int c = r / (8 * J), j = (r / 8) % J, e = r & 7;
  return q * Q + (j * 4 + c) * 8 + ((e & 3) << 1) + (e >> 2);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// D += A B, fp16 (F16) or bf16 operands, fp32 sums.
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The two e4m3 values in the low (HI false) or high half of a word as fp16.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(HI ? v >> 16 : v)));
  return h;
}

// The eight codes of a word (low nibble = code 0) as pairs (e, e + 4), e =
// 0..3, minus the zero point.  Setting the exponent of 1024 (fp16) or 128
// (bf16) above a code makes the number 1024 + code or 128 + code; the
// differences are whole numbers, exact.  In fp16 a code four bits higher up is
// 1024 + 16 code, and a fused multiply-add by 1/16 brings it down; bf16 has too
// few bits for that and shifts.
template <bool F16>
__device__ __forceinline__ void w4_pairs(uint32_t word, uint32_t zero2, uint32_t (&v)[4]) {
  if constexpr (F16) {
    const uint32_t m1032 = 0xe408e408u, m72 = 0xd480d480u, r16 = 0x2c002c00u;  // -1032, -72, 1 / 16
    const uint32_t w8 = word >> 8;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xEA;" : "=r"(v[0]) : "r"(word));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xEA;" : "=r"(v[1]) : "r"(word));
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xEA;" : "=r"(v[2]) : "r"(w8));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xEA;" : "=r"(v[3]) : "r"(w8));
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(v[0]) : "r"(m1032));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(v[1]) : "r"(r16), "r"(m72));
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(v[2]) : "r"(m1032));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(v[3]) : "r"(r16), "r"(m72));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t t;
      asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xEA;" : "=r"(t) : "r"(word >> (4 * e)));
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                                       *reinterpret_cast<const __nv_bfloat162*>(&zero2));
      v[e] = *reinterpret_cast<const uint32_t*>(&d);
    }
  }
}

template <int THREADS>
__device__ __forceinline__ void bar_consumers() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// The ring's barriers: a stage is full once its weights' bytes and the arrivals
// of the feeder warp that wrote its rows are there, empty once every warp of
// the team that took it is through.
struct StreamRing {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int abort;
  int last;  // of an arrival count (finish a shared strip)
  __device__ void init() {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&full[i], 1 + 32);
      mbar_init(&empty[i], kStreamWarps);
    }
    abort = 0;
    fence_mbarrier_init();
  }
  __device__ bool aborted() const { return *reinterpret_cast<const volatile int*>(&abort); }
  // A wait gave up: every later wait of the CTA ends at once.
  __device__ void give_up(int32_t* err) {
    if (!aborted()) {
      *reinterpret_cast<volatile int*>(&abort) = 1;
      atomicOr(err, MOE_DEV_WAIT_TIMEOUT);
    }
  }
};

// Position in a ring of n slots.
struct RingPos {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) {
      at = 0;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ void skip(int by, int n) {  // by <= n
    at += by;
    if (at >= n) {
      at -= n;
      phase ^= 1u;
    }
  }
};

// After an abort, by the producer: copies still in flight land before the CTA
// exits.  `pos` is the slot after the last one filled.
__device__ __forceinline__ void drain_ring(StreamRing* r, RingPos pos, int n) {
  for (int i = 0; i < n; ++i) {
    if (pos.at == 0) {
      pos.at = n - 1;
      pos.phase ^= 1u;
    } else {
      --pos.at;
    }
    mbar_wait_drain(&r->full[pos.at], pos.phase);
  }
  drain_grace();
}

// fp32 as the sum of two bf16 (16 significant bits); an infinity keeps a zero
// low part so that their sum is not a NaN.
__device__ __forceinline__ void split_bf16(float v, __nv_bfloat16& hi, __nv_bfloat16& lo) {
  hi = __float2bfloat16_rn(v);
  const float h = __bfloat162float(hi);
  lo = isinf(h) ? __float2bfloat16_rn(0.0f) : __float2bfloat16_rn(v - h);
}

// ------------------------------------------------------------ work of a CTA
// N equal chunks over min(G, N) CTAs: CTA b takes [N b / Gp, N (b + 1) / Gp).
struct Split {
  long long N;
  int Gp;
};
__host__ __device__ __forceinline__ Split make_split(long long N, int G) {
  return Split{N, static_cast<int>(N < G ? N : G)};
}
__host__ __device__ __forceinline__ long long split_lo(const Split& s, int b) {
  if (s.N == 0) return 0;
  return b >= s.Gp ? s.N : s.N * b / s.Gp;
}
// the CTA of chunk q
__host__ __device__ __forceinline__ int split_cta(const Split& s, long long q) {
  const unsigned long long v = static_cast<unsigned long long>(q + 1) * s.Gp - 1;
  if ((v >> 32) == 0 && (s.N >> 32) == 0)
    return static_cast<int>(static_cast<uint32_t>(v) / static_cast<uint32_t>(s.N));
  return static_cast<int>(v / static_cast<unsigned long long>(s.N));
}

// ------------------------------------------------------------ multiply a stage
// [.., K, N] weights: the warp's k16 of its half times NTU tiles of 8 tokens.
// acc[nt][mt] holds columns (2 KIND-dependent widths) as kn_col() says.
template <int KIND, int NT, bool HILO>
__device__ __forceinline__ void stage_mma_kn(uint32_t stage, uint32_t bbuf, uint32_t lo_off, int warp,
                                             int lane, int ntu,
                                             float (&acc)[NT][StreamTraits<KIND, 0>::MT][4]) {
  using Tr = StreamTraits<KIND, 0>;
  const int g = lane >> 2, c = lane & 3, half = warp & 1, kw = warp >> 1;
  // rows 2c, 2c+1, 2c+8, 2c+9 of the k16: eight lanes of a load phase (two g,
  // four c) then touch eight different 16-byte columns of the swizzled box
  const uint32_t base = stage + half * kHalfBytes + (kw * 16 + 2 * c) * 128;
  const uint32_t x0 = static_cast<uint32_t>(g ^ (2 * c)) << 4;
  const uint32_t x1 = static_cast<uint32_t>(g ^ (2 * c + 1)) << 4;
  const uint4 w0 = lds128(base + x0), w1 = lds128(base + 128 + x1);
  const uint4 w2 = lds128(base + 1024 + x0), w3 = lds128(base + 1024 + 128 + x1);
  const uint32_t ba = bbuf + g * Tr::PITCH + kw * 32 + c * 8;
  uint2 b[NT], bl[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    if (nt < ntu) {
      b[nt] = lds64(ba + nt * 8 * Tr::PITCH);
      if (HILO) bl[nt] = lds64(ba + nt * 8 * Tr::PITCH + lo_off);
    }
  const uint32_t r0[4] = {w0.x, w0.y, w0.z, w0.w}, r1[4] = {w1.x, w1.y, w1.z, w1.w};
  const uint32_t r2[4] = {w2.x, w2.y, w2.z, w2.w}, r3[4] = {w3.x, w3.y, w3.z, w3.w};
#pragma unroll
  for (int mt = 0; mt < Tr::MT; ++mt) {
    uint32_t a0, a1, a2, a3;
    if constexpr (KIND == kStreamBf16) {
      a0 = __byte_perm(r0[mt], r1[mt], 0x5410);
      a1 = __byte_perm(r0[mt], r1[mt], 0x7632);
      a2 = __byte_perm(r2[mt], r3[mt], 0x5410);
      a3 = __byte_perm(r2[mt], r3[mt], 0x7632);
    } else {
      const uint32_t sel = (mt & 1) ? 0x7362 : 0x5140;
      const uint32_t p = __byte_perm(r0[mt >> 1], r1[mt >> 1], sel);
      const uint32_t q = __byte_perm(r2[mt >> 1], r3[mt >> 1], sel);
      a0 = e4m3x2_to_f16x2<false>(p);
      a1 = e4m3x2_to_f16x2<true>(p);
      a2 = e4m3x2_to_f16x2<false>(q);
      a3 = e4m3x2_to_f16x2<true>(q);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (nt < ntu) {
        mma_16816<Tr::F16>(acc[nt][mt], a0, a1, a2, a3, b[nt].x, b[nt].y);
        if (HILO) mma_16816<Tr::F16>(acc[nt][mt], a0, a1, a2, a3, bl[nt].x, bl[nt].y);
      }
  }
}
// column (inside the half) of acc[..][mt][0..1]; [2..3] hold the next one
template <int KIND>
__device__ __forceinline__ int kn_col(int lane, int mt) {
  return (KIND == kStreamBf16 ? 8 : 16) * (lane >> 2) + 2 * mt;
}

// [.., N, K] weights: row (inside the warp's 16) of mma row g; mma row g + 8
// is that + 8.  The order makes the lanes of a load phase touch different
// 16-byte columns of the swizzled box.
template <int KIND, int GRP>
__device__ __forceinline__ int nk_row(int g) {
  if (KIND == kStreamW4 && GRP == 64) return ((g & 3) << 1) | (g >> 2);
  if (KIND == kStreamW4 && GRP == 32) return g;
  return (g >> 1) | ((g & 1) << 2);
}

// For few rows the k steps are summed in chains of their own, so that a warp has
// several multiplies in flight; the chains are added at the end of the stage.
template <int NT>
__device__ __forceinline__ void stage_mma_fp8nk(uint32_t stage, uint32_t rows, int warp, int lane, int ntu,
                                                float (&acc)[NT][1][4]) {
  using Tr = StreamTraits<kStreamFp8Nk, 0>;
  constexpr int CH = NT == 1 ? 4 : NT == 2 ? 2 : 1;
  const int g = lane >> 2, c = lane & 3;
  const int r = nk_row<kStreamFp8Nk, 0>(g);
  const uint32_t base = stage + (warp * 16 + r) * 128;
  const uint32_t ba = rows + g * Tr::PITCH + c * 16;
  float t[NT][CH][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < CH; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) t[nt][h][i] = h == 0 ? acc[nt][0][i] : 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t xo = static_cast<uint32_t>((4 * i + c) ^ r) << 4;
    const uint4 u = lds128(base + xo), v = lds128(base + 1024 + xo);
    const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[8];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        a[4 * w] = e4m3x2_to_f16x2<false>(uu[2 * h + w]);
        a[4 * w + 1] = e4m3x2_to_f16x2<false>(vv[2 * h + w]);
        a[4 * w + 2] = e4m3x2_to_f16x2<true>(uu[2 * h + w]);
        a[4 * w + 3] = e4m3x2_to_f16x2<true>(vv[2 * h + w]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (nt < ntu) {
          const uint4 b = lds128(ba + nt * 8 * Tr::PITCH + (2 * i + h) * 64);
          mma_16816<true>(t[nt][(2 * h) % CH], a[0], a[1], a[2], a[3], b.x, b.y);
          mma_16816<true>(t[nt][(2 * h + 1) % CH], a[4], a[5], a[6], a[7], b.z, b.w);
        }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = t[nt][0][i];
#pragma unroll
      for (int h = 1; h < CH; ++h) v += t[nt][h][i];
      acc[nt][0][i] = v;
    }
}

// Group scales (bf16 bits, zero point in the upper half) of a warp's 16 rows
// for one 256-k stage, spread over the four lanes of a row pair: lane c holds
// groups 2 i + c / 2 (slot i) of mma row g (even c) or g + 8 (odd c).
template <int GRP>
struct W4Scales {
  static constexpr int kSlots = 256 / GRP / 2;
  uint32_t v[kSlots];
};
// `at`: index of the lane's row's first group (-1: a row outside the matrix),
// groups = groups of a row; q0 = the stage's first group.
template <int GRP>
__device__ __forceinline__ void w4_load_scales(W4Scales<GRP>& s, const __nv_bfloat16* sc, const uint8_t* zp,
                                               long long at, int groups, int q0, int lane) {
  q0 += (lane & 3) >> 1;
#pragma unroll
  for (int i = 0; i < W4Scales<GRP>::kSlots; ++i) {
    uint32_t w = 8u << 16;
    if (at >= 0 && q0 + 2 * i < groups) {
      const long long j = at + q0 + 2 * i;
      w = __ldg(reinterpret_cast<const unsigned short*>(sc) + j) |
          (zp ? static_cast<uint32_t>(__ldg(zp + j) & 15u) << 16 : 8u << 16);
    }
    s.v[i] = w;
  }
}

template <int GRP, int NT, bool ZERO, bool F16>
__device__ __forceinline__ void stage_mma_w4(uint32_t stage, uint32_t rows, int warp, int lane, int ntu,
                                             const W4Scales<GRP>& sc, int groups_here,
                                             float (&acc)[NT][1][4]) {
  static_assert(!(ZERO && F16), "zero points come with bf16 operands");
  using Tr = StreamTraits<kStreamW4, GRP>;
  constexpr int J = GRP / 32, QB = 256 / GRP;
  constexpr int CH = NT == 1 ? 2 : 1;
  const int g = lane >> 2, c = lane & 3;
  const int r = nk_row<kStreamW4, GRP>(g);
  const uint32_t base = stage + (warp * 16 + r) * 128;
  const uint32_t ba = rows + g * Tr::PITCH + c * 16;
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    if (q >= groups_here) break;
    uint32_t wa[J], wb[J];
    if constexpr (GRP == 128) {
      const uint32_t xo = static_cast<uint32_t>((4 * q + c) ^ (r & 7)) << 4;
      const uint4 u = lds128(base + xo), v = lds128(base + 1024 + xo);
      wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
      wb[0] = v.x; wb[1] = v.y; wb[2] = v.z; wb[3] = v.w;
    } else if constexpr (GRP == 64) {
      const uint32_t xo = (static_cast<uint32_t>((2 * q + (c >> 1)) ^ (r & 7)) << 4) + (c & 1) * 8;
      const uint2 u = lds64(base + xo), v = lds64(base + 1024 + xo);
      wa[0] = u.x; wa[1] = u.y;
      wb[0] = v.x; wb[1] = v.y;
    } else {
      const uint32_t xo = (static_cast<uint32_t>(q ^ (r & 7)) << 4) + c * 4;
      wa[0] = lds32(base + xo);
      wb[0] = lds32(base + 1024 + xo);
    }
    const int from = (lane & ~3);
    const uint32_t s0 = __shfl_sync(0xffffffffu, sc.v[q >> 1], from | ((2 * q) & 3));
    const uint32_t s1 = __shfl_sync(0xffffffffu, sc.v[q >> 1], from | ((2 * q + 1) & 3));
    uint32_t z0 = 0x43084308u, z1 = 0x43084308u;  // 128 + 8
    if (ZERO) {
      z0 = s0 >> 16;
      z1 = s1 >> 16;
      z0 = 0x43004300u | z0 | (z0 << 16);
      z1 = 0x43004300u | z1 | (z1 << 16);
    }
    // for few rows the two halves of a word are summed in chains of their own
    float part[NT][CH][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < CH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[nt][h][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint32_t a[4], b[4];
      w4_pairs<F16>(wa[j], z0, a);
      w4_pairs<F16>(wb[j], z1, b);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (nt < ntu) {
          const uint4 x = lds128(ba + nt * 8 * Tr::PITCH + (q * J + j) * 64);
          mma_16816<F16>(part[nt][0], a[0], b[0], a[1], b[1], x.x, x.y);
          mma_16816<F16>(part[nt][CH - 1], a[2], b[2], a[3], b[3], x.z, x.w);
        }
    }
    const float f0 = __uint_as_float(s0 << 16), f1 = __uint_as_float(s1 << 16);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (nt < ntu) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = part[nt][0][i];
          if (CH == 2) v += part[nt][CH - 1][i];
          acc[nt][0][i] = fmaf(i < 2 ? f0 : f1, v, acc[nt][0][i]);
        }
      }
  }
}

// A ring slot: a stage's weights, then its token rows; as many (an even number)
// as fit beside `other` bytes.
constexpr int kStreamSmemMax = 232448;
__host__ __device__ constexpr int stream_slot(int row_bytes) {
  return kStageBytes + (row_bytes + 1023) / 1024 * 1024;
}
__host__ __device__ constexpr int stream_stages(int slot, int other) {
  const int n = (kStreamSmemMax - 1024 - other) / slot;
  return (n > kMaxStages ? kMaxStages : n) / 2 * 2;
}

}  // namespace moe
