// Building blocks of the kernels for a few tokens (few_layer.cuh, linear_w4.cu,
// linear_w4_wide.cu): weights streamed once from HBM through a ring of 16 KB
// shared-memory stages that one thread fills with TMA box loads, multiplied by
// at most 16 token rows with mma.sync (m16n8k16, the weights as the 16-row
// operand and the tokens as the 8 columns).
//
// Why mma.sync and not tcgen05: at a few tokens every weight is used for a
// handful of multiply-adds, so the tensor rate is no limit (one SM's share of
// HBM, ~24 bytes a cycle, feeds one m16n8k16 every 20 to 40 cycles), while a
// tcgen05 operand has to lie in shared memory in its final type: 8- and 4-bit
// weights would be expanded to bf16 there, written and read once more.  With
// mma.sync they are expanded in the registers that the multiply reads.  (From 17
// rows on, mma.sync is the limit; linear_w4_wide.cu expands into tensor memory.)
//
// Roles of a CTA: consumer warps in one or two teams of eight (two teams take
// the stages in turn and add their sums at the end of a strip: twice the time
// per stage for the latencies of a stage's loads, conversions and multiplies),
// a producer warp (weights), feeder warps (the token rows of a stage, put
// beside its weights; the feeders take the stages in turn) and a finisher warp
// (a strip's sums to memory, so that its round trips delay no consumer).
//
// Operand types: bf16 weights are multiplied as bf16; e4m3 weights and 4-bit
// codes (exact there) as fp16, by token rows that are fp16 times a power of
// two that puts the row's largest element in [2^14, 2^15).  One conversion
// makes two e4m3 values fp16, and an fp16 row needs no second term for h.
//
// A stage is 16 KB of 128-byte rows, 128-byte swizzled:
//   [.., K, N] weights (bf16, e4m3): four boxes ("quarters") of 32 consecutive k
//     x 64 or 128 columns; warp w multiplies k 16 (w / 4) .. + 15 of quarter w % 4.
//     Neighbouring quarters are 256 bytes (gate, up) or 512 bytes (down) of a row:
//     with 128-byte pieces the same layer read HBM at 4.6 TB/s, not 6;
//   [.., N, K] weights (e4m3, 4-bit): two boxes of 64 output rows x 128 or 256
//     consecutive k; warp w owns rows 32 (w / 2) .. + 31 of the 128 and one half
//     of the k (two 16-row tiles share the token rows that it loads).
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
constexpr int kStreamWarps = 8;     // consumer warps of a team
constexpr int kStreamMaxCtas = 160; // most CTAs of a launch
constexpr int kStreamMaxRows = 32;  // most token rows of a call
constexpr int kMaxStages = 12;      // of the ring

enum StreamKind : int { kStreamBf16 = 0, kStreamFp8 = 1, kStreamFp8Nk = 2, kStreamW4 = 3 };

template <int KIND, int GRP>
struct StreamTraits {
  static constexpr bool KN = KIND == kStreamBf16 || KIND == kStreamFp8;
  static constexpr int KCH = KN ? 32 : (KIND == kStreamFp8Nk ? 128 : 256);  // k of a stage
  static constexpr int BOXES = KN ? 4 : 2;
  static constexpr int BOX_ROWS = KN ? 32 : 64;
  static constexpr int QC = KIND == kStreamFp8 ? 128 : 64;  // output columns of a box
  static constexpr int HC = QC * BOXES / 2;                 // of half the boxes (gate or up)
  static constexpr int MT = KN ? QC / 16 : 2;               // 16-column mma tiles of a warp
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

// D = A B.
template <bool F16>
__device__ __forceinline__ void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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
// few bits for that and shifts.  (Published for weights of 8 and 4 bits by Kim, Henry,
// Fahim and Hassan Awadalla, "Who Says Elephants Can't Run: Bringing Large Scale MoE
// Models into Cloud Scale Production", 2022.)
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

// The same barrier; whether any thread's v is true.
template <int THREADS>
__device__ __forceinline__ bool bar_consumers_or(bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(v)), "n"(THREADS)
      : "memory");
  return any != 0;
}

// The ring's barriers: a stage is full once its weights' bytes and the arrivals
// of the feeder warp that wrote its rows are there, empty once every warp of
// the team that took it is through.
struct StreamRing {
  uint64_t full[kMaxStages], empty[kMaxStages];
  // the two buffers of finished sums that the consumers hand to the finisher
  uint64_t red_full[2], red_empty[2];
  int abort;
  int last[2];  // whether an arrival was the last (finisher's, consumers')
  // arrivals that make a stage full (a feeder's lanes beside the producer) and empty
  __device__ void init(int consumer_warps, int filled = 1 + 32, int emptied = kStreamWarps) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&red_full[i], consumer_warps);
      mbar_init(&red_empty[i], 32);
    }
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&full[i], filled);
      mbar_init(&empty[i], emptied);
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

// Adds 1 to an arrival count (release: what this thread saw written, its own CTA's
// earlier writes before a barrier among them; acquire: what the others wrote).
__device__ __forceinline__ int arrive_acq_rel(int32_t* p) {
  int v;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

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

// Which of the two buffers the next strip's sums go to, and each one's phase.
struct RedPos {
  int at = 0;
  uint32_t bits = 0;
  __device__ __forceinline__ uint32_t phase(int buf) const { return (bits >> buf) & 1u; }
  __device__ __forceinline__ void handed(int buf) { bits ^= 1u << buf; }
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
// N units over Gp CTAs: CTA b takes [N b / Gp, N (b + 1) / Gp).  (Equal runs that cut a
// tile's sum between CTAs: Osama, Merrill, Cecka, Garland and Owens, PPoPP 2023.)
struct Split {
  long long N;
  int Gp;
};
__host__ __device__ __forceinline__ Split make_split(long long N, int G) {
  return Split{N, static_cast<int>(N < G ? N : G)};
}
// (64-bit divisions cost about 100 instructions: only where they are needed)
__host__ __device__ __forceinline__ unsigned long long div_u64(unsigned long long a, unsigned long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
__host__ __device__ __forceinline__ long long split_lo(const Split& s, int b) {
  if (s.N == 0) return 0;
  return b >= s.Gp ? s.N : static_cast<long long>(div_u64(s.N * b, s.Gp));
}
// the CTA of unit u
__host__ __device__ __forceinline__ int split_cta(const Split& s, long long u) {
  return static_cast<int>(div_u64(static_cast<unsigned long long>(u + 1) * s.Gp - 1, s.N));
}

// ------------------------------------------------------------ multiply a stage
// [.., K, N] weights: the warp's k16 of its quarter times NTU tiles of 8 tokens.
// acc[nt][mt] holds columns (2 KIND-dependent widths) as kn_col() says.
template <int KIND, int NT, bool HILO>
__device__ __forceinline__ void stage_mma_kn(uint32_t stage, uint32_t bbuf, uint32_t lo_off, int warp,
                                             int lane, int ntu,
                                             float (&acc)[NT][StreamTraits<KIND, 0>::MT][4]) {
  using Tr = StreamTraits<KIND, 0>;
  const int g = lane >> 2, c = lane & 3, kw = warp >> 2;
  // rows 2c, 2c+1, 2c+8, 2c+9 of the k16: eight lanes of a load phase (two g,
  // four c) then touch eight different 16-byte columns of the swizzled box
  const uint32_t base = stage + (warp & 3) * (kStageBytes / 4) + (kw * 16 + 2 * c) * 128;
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
// column (inside the box) of acc[..][mt][0..1]; [2..3] hold the next one
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

// For few rows the two words of eight k are summed in chains of their own, so
// that a warp has four multiplies in flight; the chains are added at the end.
template <int NT>
__device__ __forceinline__ void stage_mma_fp8nk(uint32_t stage, uint32_t rows, int warp, int lane, int ntu,
                                                float (&acc)[NT][2][4]) {
  using Tr = StreamTraits<kStreamFp8Nk, 0>;
  constexpr int CH = NT == 1 ? 2 : 1;
  const int g = lane >> 2, c = lane & 3, kh = warp & 1;
  const int r = nk_row<kStreamFp8Nk, 0>(g);
  const uint32_t base = stage + ((warp >> 1) * 32 + r) * 128 + (static_cast<uint32_t>((4 * kh + c) ^ r) << 4);
  const uint32_t ba = rows + g * Tr::PITCH + kh * 128 + c * 16;
  uint32_t w[2][2][4];  // [tile][row g, g + 8][word]
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 v = lds128(base + mt * 2048 + h * 1024);
      w[mt][h][0] = v.x; w[mt][h][1] = v.y; w[mt][h][2] = v.z; w[mt][h][3] = v.w;
    }
  float t[NT][2][4];
  if (CH == 2)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) t[nt][mt][i] = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t a[2][8];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        a[mt][4 * u] = e4m3x2_to_f16x2<false>(w[mt][0][2 * h + u]);
        a[mt][4 * u + 1] = e4m3x2_to_f16x2<false>(w[mt][1][2 * h + u]);
        a[mt][4 * u + 2] = e4m3x2_to_f16x2<true>(w[mt][0][2 * h + u]);
        a[mt][4 * u + 3] = e4m3x2_to_f16x2<true>(w[mt][1][2 * h + u]);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (nt < ntu) {
        const uint4 b = lds128(ba + nt * 8 * Tr::PITCH + h * 64);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          mma_16816<true>(acc[nt][mt], a[mt][0], a[mt][1], a[mt][2], a[mt][3], b.x, b.y);
          if (CH == 2) mma_16816<true>(t[nt][mt], a[mt][4], a[mt][5], a[mt][6], a[mt][7], b.z, b.w);
          else mma_16816<true>(acc[nt][mt], a[mt][4], a[mt][5], a[mt][6], a[mt][7], b.z, b.w);
        }
      }
  }
  if (CH == 2)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][mt][i] += t[nt][mt][i];
}

// Group scales (bf16 bits) and zero points of a warp's 32 rows and half of the k of
// one 256-k stage: lane c of a quad holds those of mma row g (even c) or g + 8 (odd
// c) of tile c / 2, a slot for each group.  As they were loaded: a conversion here
// would wait for the loads.
template <int GRP, bool ZERO>
struct W4Scales {
  static constexpr int kSlots = 128 / GRP;
  uint32_t v[kSlots], z[ZERO ? kSlots : 1];
};
// `at`: index of the lane's row's first group (-1: a row outside the matrix),
// groups = groups of a row; q0 = the first group.
template <int GRP, bool ZERO>
__device__ __forceinline__ void w4_load_scales(W4Scales<GRP, ZERO>& s, const __nv_bfloat16* sc, const uint8_t* zp,
                                               long long at, int groups, int q0) {
#pragma unroll
  for (int i = 0; i < W4Scales<GRP, ZERO>::kSlots; ++i) {
    s.v[i] = 0;
    if (ZERO) s.z[i] = 0;
    if (at >= 0 && q0 + i < groups) {
      s.v[i] = __ldg(reinterpret_cast<const unsigned short*>(sc) + at + q0 + i);
      if (ZERO) s.z[i] = __ldg(zp + at + q0 + i);
    }
  }
}

// 4-bit weights: 32 rows x 128 k of the stage.  NI tiles of eight tokens share the
// converted codes and MI tiles of 16 rows the loads of the tokens; the rest is done
// again, which saves registers.  (Groups beyond the end of a row have scale 0 and
// zero token rows.)
template <int GRP, int NT, int NI, int MI, bool ZERO, bool F16>
__device__ __forceinline__ void stage_mma_w4(uint32_t stage, uint32_t rows, int warp, int lane, int ntu,
                                             const W4Scales<GRP, ZERO>& sc, float (&acc)[NT][2][4]) {
  static_assert(!(ZERO && F16), "zero points come with bf16 operands");
  using Tr = StreamTraits<kStreamW4, GRP>;
  constexpr int J = GRP / 32, QB = 128 / GRP;
  const int g = lane >> 2, c = lane & 3, kh = warp & 1;
  const int r = nk_row<kStreamW4, GRP>(g);
  const uint32_t base = stage + ((warp >> 1) * 32 + r) * 128;
  const uint32_t ba = rows + g * Tr::PITCH + kh * 256 + c * 16;
  const int from = lane & ~3;
#pragma unroll
  for (int m0 = 0; m0 < 2; m0 += MI) {
    uint32_t w[MI][2][4];  // [tile][row g, g + 8][word of eight codes]
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = base + (m0 + m) * 2048 + h * 1024;
        if constexpr (GRP == 128) {
          const uint4 u = lds128(at + (static_cast<uint32_t>((4 * kh + c) ^ (r & 7)) << 4));
          w[m][h][0] = u.x; w[m][h][1] = u.y; w[m][h][2] = u.z; w[m][h][3] = u.w;
        } else if constexpr (GRP == 64) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint2 u = lds64(at + (static_cast<uint32_t>((4 * kh + 2 * q + (c >> 1)) ^ (r & 7)) << 4) + (c & 1) * 8);
            w[m][h][2 * q] = u.x; w[m][h][2 * q + 1] = u.y;
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[m][h][q] = lds32(at + (static_cast<uint32_t>((4 * kh + q) ^ (r & 7)) << 4) + c * 4);
        }
      }
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += NI) {
      if (n0 >= ntu) break;
#pragma unroll
      for (int q = 0; q < QB; ++q) {
        float f[MI][2];
        uint32_t z[MI][2];
#pragma unroll
        for (int m = 0; m < MI; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f[m][h] = __uint_as_float(__shfl_sync(0xffffffffu, sc.v[q], from | (2 * (m0 + m) + h)) << 16);
            z[m][h] = 0x43084308u;  // 128 + zero point
            if (ZERO) {
              const uint32_t v = __shfl_sync(0xffffffffu, sc.z[q], from | (2 * (m0 + m) + h)) & 15u;
              z[m][h] = 0x43004300u | v | (v << 16);
            }
          }
        float part[NI][MI][4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          uint32_t a[MI][4], b[MI][4];
#pragma unroll
          for (int m = 0; m < MI; ++m) {
            w4_pairs<F16>(w[m][0][q * J + j], z[m][0], a[m]);
            w4_pairs<F16>(w[m][1][q * J + j], z[m][1], b[m]);
          }
#pragma unroll
          for (int n = 0; n < NI; ++n)
            if (n0 + n < ntu) {
              const uint4 x = lds128(ba + (n0 + n) * 8 * Tr::PITCH + (q * J + j) * 64);
#pragma unroll
              for (int m = 0; m < MI; ++m) {
                if (j == 0) mma_16816_first<F16>(part[n][m], a[m][0], b[m][0], a[m][1], b[m][1], x.x, x.y);
                else mma_16816<F16>(part[n][m], a[m][0], b[m][0], a[m][1], b[m][1], x.x, x.y);
              }
#pragma unroll
              for (int m = 0; m < MI; ++m)
                mma_16816<F16>(part[n][m], a[m][2], b[m][2], a[m][3], b[m][3], x.z, x.w);
            }
        }
#pragma unroll
        for (int n = 0; n < NI; ++n)
          if (n0 + n < ntu) {
#pragma unroll
            for (int m = 0; m < MI; ++m)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[n0 + n][m0 + m][e] = fmaf(f[m][e >> 1], part[n][m][e], acc[n0 + n][m0 + m][e]);
          }
      }
    }
  }
}

// A team's sums into red[row][columns] (RP floats a row): the two warps of a team
// that hold sums of the same columns, and the teams, add theirs one after
// another, in a fixed order, with a `sync` of all of them between two.
// `before_first` runs before anything is written.
template <int KIND, int GRP, int NT, int TEAMS, int RP, typename WAIT, typename SYNC>
__device__ __forceinline__ void add_sums(float* red, int team, int warp, int lane, int ntu,
                                         const float (&acc)[NT][StreamTraits<KIND, GRP>::MT][4], WAIT before_first,
                                         SYNC sync) {
  using Tr = StreamTraits<KIND, GRP>;
  const int g = lane >> 2, c = lane & 3;
  const int mine = team * 2 + (Tr::KN ? warp >> 2 : warp & 1);
  if (mine == 0) before_first();
#pragma unroll 1
  for (int r = 0; r < 2 * TEAMS; ++r) {
    if (r > 0) sync();
    if (mine == r) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (nt < ntu) {
#pragma unroll
          for (int mt = 0; mt < Tr::MT; ++mt) {
            const int col = Tr::KN ? (warp & 3) * Tr::QC + kn_col<KIND>(lane, mt)
                                   : (warp >> 1) * 32 + mt * 16 + nk_row<KIND, GRP>(g);
            constexpr int step = Tr::KN ? 1 : 8;  // column of v[2..3] after that of v[0..1]
            float* at = red + (nt * 8 + 2 * c) * RP + col;
            const float* v = acc[nt][mt];
            if (r == 0) {
              at[0] = v[0]; at[RP] = v[1]; at[step] = v[2]; at[RP + step] = v[3];
            } else {
              at[0] += v[0]; at[RP] += v[1]; at[step] += v[2]; at[RP + step] += v[3];
            }
          }
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
