// The whole MoE layer for at most 32 tokens as one cooperative launch of one
// CTA per SM (moe_layer_few).  Phases, with a grid barrier where one needs
// another CTA's results:
//   0  router projection into fp32 planes (slices of D); x in the k order of the
//      weight layout (perm_k), zero-padded to whole stages
//   -- barrier 0
//   1  top-k softmax: every CTA for every token where the planes are small (one
//      warp per token), else CTA t for token t and barrier 1; every CTA then
//      lists the chosen experts and their rows
//   2  gate/up products: the chosen experts' (and the shared expert's) weight
//      stages, one equal run of them per CTA, so that every SM streams the same
//      number of bytes whatever the routing.  At the end of a strip of columns
//      h = act(gate) * up: for bf16 weights as a bf16 pair (hi, lo) in the k order
//      of the down weights, else in fp32 with each row's largest |h|, by which the
//      down pass's feeders bring it to fp16; of a strip that several CTAs share, the
//      one that finishes last adds the partial sums (in the order of k) and does that
//   -- barrier 2
//   3  down products, divided up the same way, into fp32 rows and the partial
//      sums of shared strips
//   -- barrier 3
//   4  out = sum_j w_j y_j + shared, one rounding
// The producer runs ahead of the barriers: the weights of the next phase are on
// their way while a barrier is waited for (160 KB per SM for bf16 and e4m3 weights, 128
// for e4m3 [N, K] and bf16 with more than eight tokens, 128 and 96 for 4-bit ones), and the shared
// expert's are brought into L2 while the routing is found out.
//
// Figures (D, E, k, I, shared I; floor: the weights' bytes at 6.8 TB/s):
//   bf16, 1 token, 2048, 128, 8, 768                35 us, floor 11
//   bf16, 8 tokens, 2816, 128, 8, 704, 2112        133 to 142, floor 100
//   e4m3, 1 token, 8192, 256, 8, 2048, 2048         92 ([N, K]), 90 ([K, N]), floor 67
//   e4m3, 16 tokens, the same                      800 ([N, K]), 783 to 830 ([K, N]), floor 764
//   4-bit, 19 tokens, 2816, 128, 8, 704, 2112      124 to 130, floor 43
//   4-bit, 1 token, 2048, 128, 8, 768               27, floor 3
// (a range: GPUs differ)
// What bounds it: HBM where a CTA has many stages and a stage's products take less
// than its bytes (697 cycles: e4m3 218 to 383, bf16 145 to 304, 4-bit 552 for eight
// rows and 724 for sixteen); else the chain of routing (7 us at one token), three
// barriers (1 us each), the hand-over of shared strips (3 us) and the last sum (2).
#pragma once

#include "stream_sm103.cuh"
#include "topk_warp.cuh"

namespace moe {

constexpr int kFewMaxPlanes = 16;
constexpr int kFewMaxR = 512;  // expanded rows: 32 tokens, 16 experts each
// Most rows of one expert that a pass over its weights multiplies; an expert with
// more rows (the shared one above 16 tokens) is listed twice and streamed twice.
// Accumulators for 32 rows would leave room for one consumer team only, which
// costs every expert more than the few long ones gain.
constexpr int kFewGroup = 16;
// Stages of a short strip (of 4-bit down products; see solo()).
constexpr int kFewShort = 3;
// Up to this many bytes of router planes every CTA reads them all (152 x 64 KB
// from L2 take about as long as one more barrier).
constexpr int kFewPlaneBytes = 65536;

struct FewParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* Wg;  // null: ids and topw are given
  const float* bias;
  const void *s13, *s2, *s13s, *s2s;  // fp32 per column (e4m3) or bf16 per group (4-bit)
  __nv_bfloat16* out;
  int32_t* err;
  uint32_t* bar;  // grid barriers: arrivals of barrier i at [8 i], all zero between launches but
                  // barrier 3's, which the next launch clears
  int32_t* cnt;   // [kStreamMaxCtas]: arrivals at the strip that CTA c begins and others share
  float* logits;
  int32_t* ids;
  float* topw;
  float* planes;       // [nplanes][T][E]
  uint16_t* xp;        // [T][Dp]: x in the weights' k order, bf16 or scaled fp16
  float* xinv;         // [T]: what undoes the scale
  void* hp;            // [R + T][Ip] h, row R + t token t of the shared expert: fp32 in natural
                       // order, or (bf16 weights) [2][R + T][Ip] bf16 hi and lo in the k order
  uint32_t* hmax;      // [R + T]: the row's largest |h| (bits of an fp32)
  float* part;         // [ctas][2][T][2 HC]: gate/up sums of shared strips
  float* prim;         // [R + T][W]: the first partial sum of every down strip of a row
  float* extra;        // [ctas][T][2 HC]: a CTA's part of a down strip begun by an earlier one
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

// One pass over weights: the shared expert's strips, then the chosen experts'
// (entry by entry), every strip C chunks (stages) long; this CTA's run of the
// chunks.  Index 0 of
// S, C, K, width: the shared expert, 1: the routed ones.
struct FewPass {
  // A chunk counts w[r] units in the split: of e4m3 and 4-bit weights, more than eight
  // rows make a chunk slower than HBM (two tiles to multiply, more rows to feed).
  Split sp;
  int w[2];
  long long lo, hi, shared;  // chunks; shared: of the shared expert (all its entries)
  int shared_entries;
  int S[2], C[2];            // strips of an expert, chunks of a strip
  int K[2], width[2];        // the reduction, the output columns (of gate and up each)
};
template <int KIND, int GRP, int NT>
struct FewSmem {
  using Tr = StreamTraits<KIND, GRP>;
  // Two consumer teams where the accumulators leave room (at most 96 registers a thread)
  static constexpr int kTeams = KIND == kStreamFp8 && NT == 2 ? 1 : 2;
  static constexpr int kCons = 32 * kStreamWarps * kTeams;  // consumer threads
  static constexpr int kFeeders = 2;                        // feeder warps
  static constexpr int kBlock = kCons + 32 + 32 * kFeeders + 32;  // + producer, feeders, finisher: 12 or 20 warps
  // token rows of a stage: bf16 weights take h as two terms
  static constexpr bool kHilo = KIND == kStreamBf16;
  static constexpr int kRows = (kHilo ? 2 : 1) * 8 * NT * Tr::PITCH;
  static constexpr int kSlot = stream_slot(kRows);
  static constexpr int kRP = 2 * Tr::HC + 4;  // floats per row of red
  // the router's partial sums take kPlanes planes of red
  static constexpr int kPlanes = NT == 1 ? 4 : 2;
  static constexpr int kRedBytes = 8 * NT * 4 * (kRP > 68 * kPlanes ? kRP : 68 * kPlanes);
  static constexpr int kRedBufs = kRedBytes > 20000 ? 1 : 2;
  struct Ctrl {
    StreamRing ring;
    int na;
    FewPass pass[2];        // gate/up, down
    int cnt[512];           // rows of an expert (many rows); expert and rank of a sorted row (few)
    int ids[kFewMaxR];      // expert of an expanded row
    float w[kFewMaxR];      // its weight
    // the chosen experts in ascending order, one entry for each group of 16 rows
    uint16_t aexp[512];     // expert of an entry
    uint16_t aoff[513];     // its first sorted position
    uint16_t amap[512];     // expert -> its first entry
    uint16_t srow[kFewMaxR + kStreamMaxRows];  // token of a row (routed in sorted order, then shared)
    uint16_t pos[kFewMaxR];   // sorted position of an expanded row
  };
  static constexpr int kOther = kRedBufs * kRedBytes + static_cast<int>(sizeof(Ctrl)) + 16;
  static constexpr int NST = stream_stages(kSlot, kOther);
  static constexpr int kBytes = 1024 + NST * kSlot + kOther;
  static_assert(NST >= 4 && NST % kFeeders == 0, "ring sizes");
  static_assert(KIND != kStreamW4 || (kTeams == 2 && kRedBufs == 2 && NST >= 2 * kFewShort), "short strips");
  static_assert(kBytes <= kStreamSmemMax, "shared memory");
};

// The first chunk that starts at unit u or later; the unit at which chunk q starts.
__device__ __forceinline__ long long few_chunk(const FewPass& f, long long u) {
  if (f.w[0] == 1) return u;
  const long long su = f.shared * f.w[0];
  return u < su ? static_cast<long long>(div_u64(u + f.w[0] - 1, f.w[0]))
                : f.shared + static_cast<long long>(div_u64(u - su + f.w[1] - 1, f.w[1]));
}
__device__ __forceinline__ long long few_unit(const FewPass& f, long long q) {
  if (f.w[0] == 1) return q;
  return q < f.shared ? q * f.w[0] : f.shared * f.w[0] + (q - f.shared) * f.w[1];
}
__device__ __forceinline__ int few_cta(const FewPass& f, long long q) { return split_cta(f.sp, few_unit(f, q)); }
template <int KIND, int GRP>
__device__ __forceinline__ FewPass few_pass(const FewParams& p, bool down, int na, int G, int b) {
  using Tr = StreamTraits<KIND, GRP>;
  FewPass f;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int I = r ? p.I : p.Is;
    f.K[r] = down ? I : p.D;
    f.width[r] = down ? p.D : I;
    const int per = down ? 2 * Tr::HC : Tr::HC;
    f.S[r] = (f.width[r] + per - 1) / per;
    f.C[r] = (f.K[r] + Tr::KCH - 1) / Tr::KCH;
  }
  f.shared_entries = p.Is > 0 ? (p.T + kFewGroup - 1) / kFewGroup : 0;
  f.shared = static_cast<long long>(f.shared_entries) * f.S[0] * f.C[0];
  f.w[0] = f.w[1] = 1;
  if (KIND != kStreamBf16 && p.T > 8 && f.shared > 0 && p.T * p.k <= 5 * na) {
    // The shared expert's entries have more than eight rows, two tiles to multiply, the
    // routed ones mostly one while they have few rows on average.  Weighed against equal
    // parts, in us (32 tokens, 4096, I 2048 or 1024, shared 2048, by rows a routed entry):
    //                       1.6 (64 experts, T 16)   4 (16 experts)   8 (8)        16 (4)
    //   4-bit, groups of 64     139 : 160             122 : 135        96 : 93      88 : 84
    //   e4m3 [N, K]             117 : 140             109 : 123        92 : 85      83 : 75
    //   e4m3 [K, N]             135 : 137             104 : 104        81 : 78      78 : 75
    //   bf16 (3:2)              183 : 183             152 : 152       107 : 102     85 : 83
    // (12 tokens, 4 experts, 6 rows an entry: 61.4 : 60.7, 52.0 : 52.0, 61.2 : 60.0, 65.2 :
    // 64.1).  17 tokens, whose second shared entry has one row, 128 experts, 2816: 118 : 154,
    // 120 : 142, 157 : 156.  2:1 since a team takes a short strip alone (135 -> 124 us at 19
    // tokens).
    constexpr bool nk8 = KIND == kStreamFp8Nk;
    if (KIND == kStreamW4 && down && f.C[1] <= kFewShort) f.w[0] = 2;
    else if (KIND == kStreamW4) f.w[0] = 4, f.w[1] = 3;
    else if (down) f.w[0] = nk8 ? 9 : 3, f.w[1] = nk8 ? 4 : 2;
  }
  // (at least w[0] units, so at least one chunk, for every CTA that has a part)
  f.sp.N = f.shared * f.w[0] + static_cast<long long>(na) * f.S[1] * f.C[1] * f.w[1];
  // Small layers: a CTA takes four chunks at least, or a whole short strip.  A strip
  // that CTAs share costs its last one about 4 us, as much as ten chunks take.
  const int least = f.w[0] * max(4, min(8, f.C[1]));
  f.sp.Gp = f.sp.N >= static_cast<long long>(G) * least ? G : max(1, static_cast<int>(f.sp.N) / least);
  f.lo = few_chunk(f, split_lo(f.sp, b));
  f.hi = few_chunk(f, split_lo(f.sp, b + 1));
  return f;
}
// A chunk's place: shared (r 0) or routed (r 1) expert, entry, strip, chunk of
// the strip.
struct FewAt {
  int r, a, s, kc;
  __device__ __forceinline__ FewAt(const FewPass& f, long long q) {
    r = q >= f.shared;
    if (r) q -= f.shared;
    if ((f.sp.N >> 31) == 0) {  // 32-bit divisions unless the pass is huge
      const uint32_t strip = static_cast<uint32_t>(q) / static_cast<uint32_t>(f.C[r]);
      kc = static_cast<int>(static_cast<uint32_t>(q) - strip * f.C[r]);
      a = static_cast<int>(strip / static_cast<uint32_t>(f.S[r]));
      s = static_cast<int>(strip - static_cast<uint32_t>(a) * f.S[r]);
    } else {
      const long long strip = q / f.C[r];
      kc = static_cast<int>(q - strip * f.C[r]);
      a = static_cast<int>(strip / f.S[r]);
      s = static_cast<int>(strip - static_cast<long long>(a) * f.S[r]);
    }
  }
  __device__ __forceinline__ void next_strip(const FewPass& f) {
    kc = 0;
    if (++s == f.S[r]) {
      s = 0;
      if (++a == f.shared_entries && !r) {
        r = 1;
        a = 0;
      }
    }
  }
  __device__ __forceinline__ void next(const FewPass& f) {
    if (++kc == f.C[r]) next_strip(f);
  }
};

template <int KIND, int GRP, int NT>
struct Few {
  using Tr = StreamTraits<KIND, GRP>;
  using Sm = FewSmem<KIND, GRP, NT>;
  using Ctrl = typename Sm::Ctrl;
  static constexpr int CT = Sm::kCons;

  static __device__ __forceinline__ void bar() { bar_consumers<CT>(); }
  // An entry's rows: the first one's place in the row arrays (routed rows in
  // sorted order, then the shared expert's), and how many.
  static __device__ __forceinline__ int row_first(const FewParams& p, const Ctrl* ctl, const FewAt& at) {
    return at.r ? ctl->aoff[at.a] : p.T * p.k + at.a * kFewGroup;
  }
  static __device__ __forceinline__ int row_count(const FewParams& p, const Ctrl* ctl, const FewAt& at) {
    return at.r ? ctl->aoff[at.a + 1] - ctl->aoff[at.a] : min(kFewGroup, p.T - at.a * kFewGroup);
  }

  // Grid barrier i, by the consumers.  One CTA clears the arrivals of `clear`,
  // a barrier that every CTA has left.
  static __device__ __forceinline__ void grid_sync(const FewParams& p, StreamRing* ring, int i, int clear) {
    bar();
    if (threadIdx.x == 0 && !ring->aborted()) {
      uint32_t* at = p.bar + 8 * i;
      asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(at) : "memory");
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t n = 1;; ++n) {
        uint32_t now;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(at) : "memory");
        if (now == gridDim.x) break;
        if ((n & 63u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
          ring->give_up(p.err);
          break;
        }
      }
      if (blockIdx.x == 0 && clear >= 0) *reinterpret_cast<volatile uint32_t*>(p.bar + 8 * clear) = 0;
      if (blockIdx.x == 0 && i == 2) *reinterpret_cast<volatile uint32_t*>(p.bar + 8) = 0;
    }
    bar();
  }

  // ---------------------------------------------------------------- producer
  template <bool DOWN>
  static __device__ __forceinline__ bool produce(const CUtensorMap* routed, const CUtensorMap* shared,
                                                 const FewPass& f, const Ctrl* ctl, StreamRing* r, uint8_t* ring,
                                                 RingPos& pos, uint64_t policy) {
    if (f.lo >= f.hi) return true;
    FewAt at(f, f.lo);
#pragma unroll 1
    for (int left = static_cast<int>(f.hi - f.lo); left > 0; --left) {
      if (!mbar_wait(&r->empty[pos.at], pos.phase ^ 1u, &r->abort)) return false;
      uint64_t* full = &r->full[pos.at];
      uint8_t* dst = ring + pos.at * Sm::kSlot;
      const CUtensorMap* m = at.r ? routed : shared;
      const int e = at.r ? ctl->aexp[at.a] : 0;
      mbar_arrive_expect_tx(full, kStageBytes);
#pragma unroll
      for (int h = 0; h < Tr::BOXES; ++h) {
        uint8_t* d = dst + h * (kStageBytes / Tr::BOXES);
        if (Tr::KN) {
          if (DOWN) tma_load_3d(d, m, full, at.s * 2 * Tr::HC + h * Tr::QC, at.kc * Tr::KCH, e, policy);
          else tma_load_4d(d, m, full, at.s * Tr::HC + (h & 1) * Tr::QC, h >> 1, at.kc * Tr::KCH, e, policy);
        } else {
          if (DOWN) tma_load_3d(d, m, full, at.kc * 128, at.s * 128 + h * 64, e, policy);
          else tma_load_4d(d, m, full, at.kc * 128, at.s * 64, h, e, policy);
        }
      }
      pos.next(Sm::NST);
      at.next(f);
    }
    return true;
  }

  // While the routing is found out: this CTA's share of the shared expert's
  // weights into L2, as much as that holds.
  template <bool DOWN>
  static __device__ __forceinline__ void prefetch_shared(const FewParams& p, const CUtensorMap* m, int b, int G,
                                                         int most) {
    FewPass f = few_pass<KIND, GRP>(p, DOWN, 0, G, b);
    const Split sp = make_split(static_cast<long long>(f.S[0]) * f.C[0], G);
    f.lo = split_lo(sp, b);
    f.hi = split_lo(sp, b + 1);
    if (f.lo >= f.hi) return;
    FewAt at(f, f.lo);
#pragma unroll 1
    for (int left = min(most, static_cast<int>(f.hi - f.lo)); left > 0; --left) {
#pragma unroll
      for (int h = 0; h < Tr::BOXES; ++h) {
        if (Tr::KN) {
          if (DOWN) tma_prefetch_l2_3d(m, at.s * 2 * Tr::HC + h * Tr::QC, at.kc * Tr::KCH, 0);
          else tma_prefetch_l2_4d(m, at.s * Tr::HC + (h & 1) * Tr::QC, h >> 1, at.kc * Tr::KCH, 0);
        } else {
          if (DOWN) tma_prefetch_l2_3d(m, at.kc * 128, at.s * 128 + h * 64, 0);
          else tma_prefetch_l2_4d(m, at.kc * 128, at.s * 64, h, 0);
        }
      }
      at.next(f);
    }
  }

  // ------------------------------------------------------------------ feeder
  // e such that 2^e puts a row with largest element `bits` in [2^14, 2^15): 0 for
  // rows of zeros, at most 100 (a row below 2^-86 keeps fewer bits).  A row with
  // an infinity or NaN takes -113, which no finite element overflows at.
  static __device__ __forceinline__ int row_exp(uint32_t bits) {
    const int e = static_cast<int>(bits >> 23);
    return bits == 0 ? 0 : max(-113, min(100, 141 - e));
  }
  static __device__ __forceinline__ float exp2_int(int e) { return __int_as_float((127 + e) << 23); }

  // The token rows of the run's chunks that this feeder warp takes: those of every
  // second slot (always the same slots, so that a wait cannot mistake a fill for the
  // one before).  n rows x KCH inputs, 8 inputs a lane.
  template <bool DOWN>
  static __device__ __forceinline__ bool feed(const FewParams& p, const FewPass& f, Ctrl* ctl, uint8_t* ring,
                                              RingPos& ring_pos, int me, int lane) {
    constexpr int P = Tr::KCH / 8;  // pieces of a row
    static_assert(Sm::kFeeders == 2 && Sm::NST % 2 == 0, "slots of a feeder");
    if (f.lo >= f.hi) return true;
    const int total = static_cast<int>(f.hi - f.lo), skip = (ring_pos.at + me) & 1;
    RingPos pos = ring_pos;
    if (skip) pos.next(Sm::NST);
    ring_pos.skip(total % Sm::NST, Sm::NST);
    ring_pos.phase ^= (total / Sm::NST) & 1;
    if (skip >= total) return true;
    FewAt at(f, f.lo + skip);
    if constexpr (DOWN && !Sm::kHilo) {
      // fp32 h to scaled fp16, in the weights' k order; the first pieces of the
      // feeder's next chunk are loaded before it waits for that chunk's slot
      constexpr int U = P == 4 ? 2 : 4;  // pieces in flight (eight spill: slower)
      float4 a[U], b[U];
      uint32_t mx[U];
      auto load = [&](const FewAt& x, int first, int n, int i0) {
        const int k_end = f.K[x.r] - x.kc * Tr::KCH;  // inputs of this chunk (zeros beyond)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + 32 * u, pc = i % P, row = i / P;
          a[u] = b[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          mx[u] = 0;
          if (i < n * P && pc * 8 < k_end) {
            const int r = first + row;
            const float4* src = reinterpret_cast<const float4*>(
                static_cast<const float*>(p.hp) + static_cast<size_t>(r) * p.Ip + x.kc * Tr::KCH + pc * 8);
            a[u] = src[0];  // (through L1: every strip takes the same rows)
            b[u] = src[1];
            mx[u] = p.hmax[r];
          }
        }
      };
      auto store = [&](uint8_t* rows, int n, int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + 32 * u, pc = i % P, row = i / P;
          if (i < n * P) {
            const float sc = exp2_int(row_exp(mx[u]));
            const float v[8] = {a[u].x, a[u].y, a[u].z, a[u].w, b[u].x, b[u].y, b[u].z, b[u].w};
            uint8_t* d = rows + row * Tr::PITCH;
            auto pair = [&](int j0, int j1) {
              const __half2 h = __floats2half2_rn(v[j0] * sc, v[j1] * sc);
              return *reinterpret_cast<const uint32_t*>(&h);
            };
            const int at8 = perm_k<KIND, GRP>(pc * 8) * 2;
            if constexpr (Tr::KN) {  // pairs go to every other word
#pragma unroll
              for (int j = 0; j < 8; j += 2) *reinterpret_cast<uint32_t*>(d + at8 + j * 4) = pair(j, j + 1);
            } else if constexpr (KIND == kStreamW4) {
              *reinterpret_cast<uint4*>(d + at8) = make_uint4(pair(0, 4), pair(1, 5), pair(2, 6), pair(3, 7));
            } else {
              // (pieces of 16 inputs: the second one lies 64 bytes on)
              *reinterpret_cast<uint4*>(d + at8) = make_uint4(pair(0, 1), pair(2, 3), pair(4, 5), pair(6, 7));
            }
          }
        }
      };
      int first = row_first(p, ctl, at), n = row_count(p, ctl, at);
      load(at, first, n, lane);
#pragma unroll 1
      for (int left = total - skip; left > 0; left -= 2) {
        if (!mbar_wait(&ctl->ring.empty[pos.at], pos.phase ^ 1u, &ctl->ring.abort)) return false;
        uint8_t* rows = ring + pos.at * Sm::kSlot + kStageBytes;
        store(rows, n, lane);
#pragma unroll 1
        for (int i0 = lane + 32 * U; i0 - lane < n * P; i0 += 32 * U) {
          load(at, first, n, i0);
          store(rows, n, i0);
        }
        mbar_arrive(&ctl->ring.full[pos.at]);
        pos.skip(2, Sm::NST);
        if (left > 2) {
          at.next(f);
          at.next(f);
          first = row_first(p, ctl, at);
          n = row_count(p, ctl, at);
          load(at, first, n, lane);
        }
      }
    } else {
#pragma unroll 1
      for (int left = total - skip; left > 0; left -= 2) {
        if (!mbar_wait(&ctl->ring.empty[pos.at], pos.phase ^ 1u, &ctl->ring.abort)) return false;
        const int first = row_first(p, ctl, at), n = row_count(p, ctl, at);
        const uint32_t dst = smem_u32(ring) + pos.at * Sm::kSlot + kStageBytes;
        const size_t plane = static_cast<size_t>(p.T * p.k + p.T) * p.Ip;
        for (int i = lane; i < n * P; i += 32) {
          const int pc = i % P, row = i / P;
          const int src = DOWN ? first + row : ctl->srow[first + row];
          const uint16_t* g = (DOWN ? static_cast<const uint16_t*>(p.hp) : p.xp) +
                              static_cast<size_t>(src) * (DOWN ? p.Ip : p.Dp) + at.kc * Tr::KCH + pc * 8;
          const uint32_t d = dst + row * Tr::PITCH + pc * 16;
          cp_async_16(d, g, 16);
          if (DOWN) cp_async_16(d + 8 * NT * Tr::PITCH, g + plane, 16);
        }
        cp_async_mbar_arrive_noinc(&ctl->ring.full[pos.at]);
        pos.skip(2, Sm::NST);
        if (left > 2) {
          at.next(f);
          at.next(f);
        }
      }
    }
    return true;
  }

  // --------------------------------------------------------------- consumers
  // Where the partial sums of shared strips of gate/up are: CTA `cta`'s part of
  // a strip begun earlier (which 0) or of one it leaves unfinished (1).
  static __device__ __forceinline__ float* part_at(const FewParams& p, int cta, int which) {
    return p.part + (static_cast<size_t>(cta) * 2 + which) * p.T * 2 * Tr::HC;
  }

  // A finished gate/up strip (its sums by sum(row, column)) to h rows, two columns
  // a thread, four times at once.  bf16 weights: the last strip also zeroes the
  // row up to the end of the down pass's last stage.
  template <int THREADS, typename SUM>
  static __device__ __forceinline__ void finish_h(const FewParams& p, const FewPass& f, const Ctrl* ctl,
                                                  const FewAt& at, int n, int i0, SUM sum) {
    constexpr int U = 4, per = Tr::HC / 2;  // per: threads of a row, whole warps
    const int first = row_first(p, ctl, at), c0 = at.s * Tr::HC, width = f.width[at.r];
    const float* sc = static_cast<const float*>(at.r ? p.s13 : p.s13s) +
                      (at.r ? static_cast<size_t>(ctl->aexp[at.a]) * 2 * width : 0);
#pragma unroll 1
    for (; i0 < n * per; i0 += U * THREADS) {
      float2 g[U], u[U], sg[U], su[U];
      float inv[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * THREADS, row = i / per, k = c0 + (i % per) * 2;
        g[j] = u[j] = make_float2(0.0f, 0.0f);
        sg[j] = su[j] = make_float2(1.0f, 1.0f);
        inv[j] = 1.0f;
        if (i < n * per && k < width) {
          g[j] = sum(row, k - c0);
          u[j] = sum(row, k - c0 + Tr::HC);
          if constexpr (Tr::F16) inv[j] = __ldcg(p.xinv + ctl->srow[first + row]);
          if constexpr (KIND == kStreamFp8 || KIND == kStreamFp8Nk) {
            sg[j] = __ldg(reinterpret_cast<const float2*>(sc + k));
            su[j] = __ldg(reinterpret_cast<const float2*>(sc + width + k));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * THREADS, row = i / per, k = c0 + (i % per) * 2;
        if (i >= n * per) break;  // (whole warps)
        float2 h;
        h.x = few_act(g[j].x * inv[j] * sg[j].x, u[j].x * inv[j] * su[j].x, p.act);
        h.y = few_act(g[j].y * inv[j] * sg[j].y, u[j].y * inv[j] * su[j].y, p.act);
        const size_t o = static_cast<size_t>(first + row) * p.Ip;
        if constexpr (Tr::F16) {
          if (k < width) *reinterpret_cast<float2*>(static_cast<float*>(p.hp) + o + k) = h;
          // the bits of non-negative floats order as the floats do (NaN highest);
          // a warp's lanes are all of one row
          const uint32_t m = __reduce_max_sync(0xffffffffu, max(__float_as_uint(h.x) & 0x7fffffffu,
                                                                __float_as_uint(h.y) & 0x7fffffffu));
          if ((threadIdx.x & 31) == 0) atomicMax(p.hmax + first + row, m);
        } else if (k < p.Ip) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.hp) + o + perm_k<KIND, GRP>(k);
          __nv_bfloat162 hi, lo;
          split_bf16(h.x, hi.x, lo.x);
          split_bf16(h.y, hi.y, lo.y);
          *reinterpret_cast<__nv_bfloat162*>(dst) = hi;
          *reinterpret_cast<__nv_bfloat162*>(dst + static_cast<size_t>(p.T * p.k + p.T) * p.Ip) = lo;
        }
      }
    }
  }

  // One strip's sums (red), or this CTA's part of them, by THREADS threads (the
  // finisher warp, or all consumers): down strips become fp32 rows; gate/up strips
  // become h, those that several CTAs share by the one that arrives last.
  template <bool DOWN, int THREADS>
  static __device__ __noinline__ void finish_strip(const FewParams& p, const FewPass& f, Ctrl* ctl, const float* red,
                                                   FewAt at, int end, long long q0, int b, int i0) {
    constexpr int RP = Sm::kRP, Q = 2 * Tr::HC / 4;
    const int n = row_count(p, ctl, at);
    const bool begun_earlier = at.kc != 0;
    if (!DOWN && end == f.C[at.r] && !begun_earlier) {  // the whole strip is this CTA's
      finish_h<THREADS>(p, f, ctl, at, n, i0,
                        [&](int row, int col) { return *reinterpret_cast<const float2*>(red + row * RP + col); });
      return;
    }
    float* dst;
    size_t pitch = 2 * Tr::HC;
    if (!DOWN) {
      dst = part_at(p, b, begun_earlier ? 0 : 1);
    } else if (begun_earlier) {
      dst = p.extra + static_cast<size_t>(b) * p.T * 2 * Tr::HC;
    } else {
      dst = p.prim + static_cast<size_t>(row_first(p, ctl, at)) * p.W + static_cast<size_t>(at.s) * 2 * Tr::HC;
      pitch = p.W;
    }
#pragma unroll 2
    for (int i = i0; i < n * Q; i += THREADS) {
      const int row = i / Q, col = (i % Q) * 4;
      *reinterpret_cast<float4*>(dst + row * pitch + col) = *reinterpret_cast<const float4*>(red + row * RP + col);
    }
    if (DOWN) return;
    const int c0 = few_cta(f, q0), c1 = few_cta(f, q0 + f.C[at.r] - 1);
    int last = 0;
    if (THREADS == 32) {
      __syncwarp();
      if (i0 == 0) last = arrive_acq_rel(p.cnt + c0) == c1 - c0;
      last = __shfl_sync(0xffffffffu, last, 0);
      __syncwarp();  // what lane 0 acquired
    } else {
      bar();
      if (i0 == 0) ctl->ring.last[1] = arrive_acq_rel(p.cnt + c0) == c1 - c0;
      bar();
      last = *reinterpret_cast<volatile int*>(&ctl->ring.last[1]);
    }
    if (!last) return;
    const size_t step = static_cast<size_t>(2) * p.T * 2 * Tr::HC;  // from a CTA's parts to the next one's
    const float* head = part_at(p, c0, 1);
    const float* rest = part_at(p, c0 + 1, 0);
    finish_h<THREADS>(p, f, ctl, at, n, i0, [&](int row, int col) {
      const size_t o = static_cast<size_t>(row) * 2 * Tr::HC + col;
      // c1 > c0; three parts in flight
      float2 v = __ldcg(reinterpret_cast<const float2*>(head + o));
      const float2 w = __ldcg(reinterpret_cast<const float2*>(rest + o));
      float2 x = make_float2(0.0f, 0.0f);
      if (c1 > c0 + 1) x = __ldcg(reinterpret_cast<const float2*>(rest + step + o));
      v.x = v.x + w.x + x.x;
      v.y = v.y + w.y + x.y;
#pragma unroll 1
      for (int cta = c0 + 3; cta <= c1; ++cta) {
        const float2 m = __ldcg(reinterpret_cast<const float2*>(rest + (cta - c0 - 1) * step + o));
        v.x += m.x;
        v.y += m.y;
      }
      return v;
    });
  }

  // Short strips of 4-bit down products: a strip for each team, so that neither waits
  // for the other at its end (of three stages one team would have two, the other one).
  // Both teams' strips are in the ring at a time.  19 tokens: 135 us, not 145.
  //
  // A wait for a slot's fill n by parity takes fill n - 2's completion for its own while
  // fill n - 1 is under way.  Strips of both teams meet at barriers, so that a team knows
  // the other's stages to have landed, and inside a strip a slot (their number is even)
  // stays with one team; one team's stages of solo strips say nothing about the other's,
  // and copies land in any order.  So where a slot's last fill was the other team's
  // (unseen()), a team first waits for that one to be emptied, as the producer did: the
  // barrier's phase n - 1 cannot be mistaken, since phase n needs this warp's own arrival,
  // and phase n - 2 is over because the team has seen a stage at most 2 kFewShort <= NST
  // before this one.  (A wait at each stage would cost 19 tokens 2 us more.)
  static __device__ __forceinline__ bool solo(bool down, const FewPass& f, const FewAt& at) {
    return KIND == kStreamW4 && down && f.C[at.r] <= kFewShort;
  }
  // Which stages of a solo strip of C (a bit each) lie in slots that the other team filled
  // last: NST stages back is an odd number of strips back.
  static __host__ __device__ constexpr int unseen(int C) {
    int m = 0;
    for (int j = 0; j < C; ++j) m |= (((Sm::NST - j + C - 1) / C) & 1) << j;
    return m;
  }

  // Who finishes a strip: all consumers (of a solo strip: its team) the run's last one, when they have nothing
  // else to do, and shared ones of more than two rows, whose parts one warp would
  // add for tens of microseconds; the finisher warp the others.
  static __device__ __forceinline__ bool by_consumers(const FewParams& p, const FewPass& f, const Ctrl* ctl,
                                                      const FewAt& at, int chunks, int left) {
    return left == 0 || (chunks != f.C[at.r] && row_count(p, ctl, at) > 2);
  }

  // The finisher's part of a pass: the sums of the strips that the consumers hand
  // over.
  template <bool DOWN>
  static __device__ __forceinline__ void finish(const FewParams& p, const FewPass& f, Ctrl* ctl, const float* red0,
                                                RedPos& rpos, int b, int lane) {
    if (f.lo >= f.hi) return;
    FewAt at(f, f.lo);
    int left = static_cast<int>(f.hi - f.lo), turn = 0;
#pragma unroll 1
    for (;;) {
      const int chunks = min(f.C[at.r] - at.kc, left), end = at.kc + chunks;
      left -= chunks;
      int buf = rpos.at;
      if (solo(DOWN, f, at)) {
        buf = turn;
        turn ^= 1;
      }
      if (by_consumers(p, f, ctl, at, chunks, left)) {
        if (left == 0) break;
        at.next_strip(f);
        continue;
      }
      if (!mbar_wait(&ctl->ring.red_full[buf], rpos.phase(buf), &ctl->ring.abort)) ctl->ring.give_up(p.err);
      __syncwarp();
      finish_strip<DOWN, 32>(p, f, ctl, red0 + buf * (Sm::kRedBytes / 4), at, end, f.hi - left - end, b, lane);
      __syncwarp();
      mbar_arrive(&ctl->ring.red_empty[buf]);
      rpos.handed(buf);
      rpos.at = (buf + 1) % Sm::kRedBufs;
      at.next_strip(f);
    }
  }

  // fp32 h rows of the run's first strip, one line a thread.
  static __device__ __forceinline__ void prefetch_h(const FewParams& p, const FewPass& f, const Ctrl* ctl) {
    if (f.lo >= f.hi) return;
    const FewAt at(f, f.lo);
    const int r0 = row_first(p, ctl, at), n = row_count(p, ctl, at);
    const int lines = (f.K[at.r] + 31) / 32, i = threadIdx.x;
    if (i < n * lines)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const float*>(p.hp) +
                                                    static_cast<size_t>(r0 + i / lines) * p.Ip + (i % lines) * 32));
  }

  template <bool DOWN>
  static __device__ __forceinline__ void consume(const FewParams& p, const FewPass& f, Ctrl* ctl, uint32_t ring,
                                                 float* red0, RingPos& ring_pos, RedPos& rpos, int b) {
    if (f.lo >= f.hi) return;
    const int tid = threadIdx.x, team = Sm::kTeams == 1 ? 0 : tid / (32 * kStreamWarps);
    const int warp = (tid >> 5) % kStreamWarps, lane = tid & 31;
    [[maybe_unused]] const int g = lane >> 2, c = lane & 3;
    constexpr uint32_t kLo = 8 * NT * Tr::PITCH;
    FewAt at(f, f.lo);
    int left = static_cast<int>(f.hi - f.lo), turn = 0;  // turn: the team of the next solo strip

    // 4-bit weights: the lane's row of group scales; a strip's first ones are loaded
    // while the strip before it is summed up
    [[maybe_unused]] W4Scales<GRP == 0 ? 128 : GRP, false> sc0, sc1;
    [[maybe_unused]] const __nv_bfloat16* sbase = nullptr;
    [[maybe_unused]] long long srow = 0;
    [[maybe_unused]] int groups = 0;
    auto scales = [&](auto& dst, int kc) {
      if constexpr (KIND == kStreamW4)
        w4_load_scales<GRP, false>(dst, sbase, nullptr, srow, groups, kc * (256 / GRP) + (warp & 1) * (128 / GRP));
    };
    auto first_scales = [&](const FewAt& x) {
      if constexpr (KIND == kStreamW4) {
        // the lane's row: tile c / 2, row g or g + 8; rows 64 on of a gate/up stage are up rows
        const int half = DOWN ? 0 : warp >> 2;
        const int l = x.s * (DOWN ? 128 : 64) + ((warp >> 1) & (DOWN ? 3 : 1)) * 32 + (c >> 1) * 16 +
                      nk_row<KIND, GRP>(g) + (c & 1) * 8;
        const long long e = x.r ? ctl->aexp[x.a] : 0;
        sbase = static_cast<const __nv_bfloat16*>(DOWN ? (x.r ? p.s2 : p.s2s) : (x.r ? p.s13 : p.s13s));
        groups = f.K[x.r] / GRP;
        srow = l < f.width[x.r] ? ((e * (DOWN ? 1 : 2) + half) * f.width[x.r] + l) * groups : -1;
        const bool alone = solo(DOWN, f, x);
        scales(sc0, x.kc + (alone ? 0 : team));
        scales(sc1, x.kc + (alone ? 1 : team + Sm::kTeams));
      }
    };
    if (solo(DOWN, f, at) && team == 1) {
      const int skip = f.C[at.r] - at.kc;
      FewAt x = at;
      x.next_strip(f);
      if (left > skip) first_scales(x);
    } else {
      first_scales(at);
    }

    // routed strips behind solo ones of the shared expert: any slot may be unseen
    [[maybe_unused]] const bool behind = solo(DOWN, f, at) && at.r == 0;
    float acc[NT][Tr::MT][4];
    while (left > 0) {  // a strip, or this CTA's part of it
      const bool alone = solo(DOWN, f, at);
      const bool mine = !alone || turn == team;
      const int stride = alone ? 1 : Sm::kTeams, buf = alone ? turn : rpos.at;
      const int chunks = min(f.C[at.r] - at.kc, left), end = at.kc + chunks;
      RingPos pos = ring_pos;
      ring_pos.skip(chunks % Sm::NST, Sm::NST);
      ring_pos.phase ^= (chunks / Sm::NST) & 1;
      left -= chunks;
      turn ^= alone;
      const bool by_all = by_consumers(p, f, ctl, at, chunks, left);
      if (mine) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < Tr::MT; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[i][j][t] = 0.0f;
        const int ntu = (row_count(p, ctl, at) + 7) >> 3;
        if (!alone && team) pos.next(Sm::NST);
        if constexpr (KIND == kStreamW4 && DOWN) {
          constexpr int m1 = unseen(1), m2 = unseen(2), m3 = unseen(3);
          static_assert(kFewShort == 3 && Sm::NST >= 2 * kFewShort, "solo strips");
          if (alone && !(behind && at.r)) {
            const int C = f.C[at.r];
            const uint32_t mine = ((1u << chunks) - 1u) << at.kc, other = (C == 1 ? m1 : C == 2 ? m2 : m3) & mine;
            if (other) {  // the last of them: the other team emptied the ones before it earlier
              RingPos w = pos;
              w.skip(31 - __clz(other) - at.kc, Sm::NST);
              if (!mbar_wait(&ctl->ring.empty[w.at], w.phase ^ 1u, &ctl->ring.abort)) ctl->ring.give_up(p.err);
            }
          }
        }
        auto step = [&](auto& sc, int kc) {
          if (KIND == kStreamW4 && DOWN && behind && at.r &&
              !mbar_wait(&ctl->ring.empty[pos.at], pos.phase ^ 1u, &ctl->ring.abort))
            ctl->ring.give_up(p.err);
          if (!mbar_wait(&ctl->ring.full[pos.at], pos.phase, &ctl->ring.abort)) ctl->ring.give_up(p.err);
          __syncwarp();
          const uint32_t st = ring + pos.at * Sm::kSlot, rows = st + kStageBytes;
          // (most experts of a batch of 16 have at most eight rows: the code for one tile of
          // tokens takes three quarters of the time)
          auto& one = reinterpret_cast<float(&)[1][Tr::MT][4]>(acc[0]);
          if constexpr (Tr::KN) {
            if (NT == 1 || ntu == 1) stage_mma_kn<KIND, 1, DOWN && Sm::kHilo>(st, rows, kLo, warp, lane, 1, one);
            else stage_mma_kn<KIND, NT, DOWN && Sm::kHilo>(st, rows, kLo, warp, lane, NT, acc);
          } else if constexpr (KIND == kStreamFp8Nk) {
            if (NT == 1 || ntu == 1) stage_mma_fp8nk<1>(st, rows, warp, lane, 1, one);
            else stage_mma_fp8nk<NT>(st, rows, warp, lane, NT, acc);
          } else {
            if (NT == 1 || ntu == 1) stage_mma_w4<GRP, 1, 1, 2, false, true>(st, rows, warp, lane, 1, sc, one);
            else stage_mma_w4<GRP, NT, NT, 1, false, true>(st, rows, warp, lane, NT, sc, acc);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->ring.empty[pos.at]);
          pos.skip(stride, Sm::NST);
          scales(sc, kc + 2 * stride);
        };
#pragma unroll 1
        for (int kc = at.kc + (alone ? 0 : team); kc < end; kc += stride) {
          step(sc0, kc);
          if constexpr (KIND == kStreamW4) {
            // two by two, each with scales of its own: moving them on from one step to the
            // next would wait for the loads
            if ((kc += stride) >= end) break;
            step(sc1, kc);
          }
        }
        if (KIND == kStreamW4 && left > 0) {  // of the team's next strip
          FewAt x = at;
          x.next_strip(f);
          if (solo(DOWN, f, x) && turn != team) {
            const int skip = f.C[x.r];
            x.next_strip(f);
            if (left > skip) first_scales(x);
          } else {
            first_scales(x);
          }
        }
        // the sums over this CTA's chunks of the strip, to the finisher
        float* red = red0 + buf * (Sm::kRedBytes / 4);
        auto before_first = [&]() {
          if (!mbar_wait(&ctl->ring.red_empty[buf], rpos.phase(buf) ^ 1u, &ctl->ring.abort)) ctl->ring.give_up(p.err);
          __syncwarp();
        };
        if constexpr (KIND == kStreamW4 && DOWN) {
          if (alone) {
            auto sync = [&]() { named_bar_sync(8 + team, 32 * kStreamWarps); };
            add_sums<KIND, GRP, NT, 1, Sm::kRP>(red, 0, warp, lane, ntu, acc, before_first, sync);
            if (by_all) {
              sync();
              finish_strip<DOWN, 32 * kStreamWarps>(p, f, ctl, red, at, end, f.hi - left - end, b, tid & (32 * kStreamWarps - 1));
              sync();
            } else {
              __syncwarp();
              if (lane < 2) mbar_arrive(&ctl->ring.red_full[buf]);  // (for the other team's warp too)
            }
          }
        }
        if (!alone) {
          add_sums<KIND, GRP, NT, Sm::kTeams, Sm::kRP>(red, team, warp, lane, ntu, acc, before_first, [] { bar(); });
          if (by_all) {
            bar();
            finish_strip<DOWN, CT>(p, f, ctl, red, at, end, f.hi - left - end, b, tid);
            bar();
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->ring.red_full[buf]);
          }
        }
      }
      if (!by_all) {
        rpos.handed(buf);
        rpos.at = (buf + 1) % Sm::kRedBufs;
      }
      at.next_strip(f);
    }
  }

  // Top-k softmax of tokens t0, t0 + step, ...: the planes summed by all consumers,
  // as many tokens at a time as red holds, then a warp for each token.
  static __device__ __forceinline__ void topk(const FewParams& p, int t0, int step, bool keep_logits,
                                              int32_t* ids, float* w, float* red) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int batch = min(Sm::kRedBytes / 4 / p.E, CT / 32);
    const size_t plane = static_cast<size_t>(p.T) * p.E;
#pragma unroll 1
    for (; t0 < p.T; t0 += batch * step) {
      const int here = min(batch, (p.T - t0 + step - 1) / step);
#pragma unroll 1
      for (int i = tid; i < here * p.E; i += CT) {
        const int t = i / p.E, e = i - t * p.E;
        const float* src = p.planes + static_cast<size_t>(t0 + t * step) * p.E + e;
        float v[kFewMaxPlanes];  // all in flight
#pragma unroll
        for (int pl = 0; pl < kFewMaxPlanes; ++pl) v[pl] = pl < p.nplanes ? __ldcg(src + pl * plane) : 0.0f;
        const float bias = p.bias ? __ldg(p.bias + e) : 0.0f;
        float sum = v[0];
#pragma unroll
        for (int pl = 1; pl < kFewMaxPlanes; ++pl) sum += v[pl];
        red[i] = sum + bias;
      }
      bar();
      if (wid < here) {
        const int t = t0 + wid * step;
        const float* row = red + wid * p.E;
        float* keep = keep_logits ? p.logits + static_cast<size_t>(t) * p.E : nullptr;
        if (p.E <= 128) topk_row<4>(p, row, lane, keep, ids + t * p.k, w + t * p.k);
        else if (p.E <= 256) topk_row<8>(p, row, lane, keep, ids + t * p.k, w + t * p.k);
        else topk_row<16>(p, row, lane, keep, ids + t * p.k, w + t * p.k);
      }
      bar();
    }
  }
  template <int EPL>
  static __device__ __forceinline__ void topk_row(const FewParams& p, const float* row, int lane, float* keep,
                                                  int32_t* ids, float* w) {
    float v[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = lane + 32 * i < p.E ? row[lane + 32 * i] : 0.0f;
    warp_topk_softmax<EPL>(v, lane, p.E, p.k, p.renorm, nullptr, keep, ids, w, p.err);
  }

  // The chosen experts in ascending order and their rows in ascending order.  Few
  // rows (at most 160): every row counts the rows that come before it.
  static constexpr int kPairRows = 160;
  static __device__ __forceinline__ void build_lists_pairs(const FewParams& p, Ctrl* ctl, int tid) {
    const int R = p.T * p.k;
    if (tid < kPairRows) {  // (whole warps)
      const int e = tid < R ? ctl->ids[tid] : 0x7fffffff;
      int before = 0, same = 0;
#pragma unroll 4
      for (int r = 0; r < R; ++r) {
        const int o = ctl->ids[r];
        before += o < e;
        same += o == e && r < tid;
      }
      if (tid < R) {
        const int at = before + same;
        ctl->pos[tid] = static_cast<uint16_t>(at);
        ctl->srow[at] = static_cast<uint16_t>(tid / p.k);
        ctl->cnt[at] = e | (same << 16);  // expert and rank of the sorted row
      }
    }
    if (tid < p.T) ctl->srow[R + tid] = static_cast<uint16_t>(tid);
    bar();
    if (tid < 32) {  // an entry begins at every 16th row of an expert
      int entries = 0;
#pragma unroll 1
      for (int r0 = 0; r0 < R; r0 += 32) {
        const int at = r0 + tid, v = at < R ? ctl->cnt[at] : 1 << 16;
        const bool head = at < R && ((v >> 16) & (kFewGroup - 1)) == 0;
        const unsigned m = __ballot_sync(0xffffffffu, head);
        const int a = entries + __popc(m & ((1u << tid) - 1u));
        if (head) {
          ctl->aexp[a] = static_cast<uint16_t>(v & 0xffff);
          ctl->aoff[a] = static_cast<uint16_t>(at);
          if ((v >> 16) == 0) ctl->amap[v & 0xffff] = static_cast<uint16_t>(a);
        }
        entries += __popc(m);
      }
      if (tid == 0) {
        ctl->na = entries;
        ctl->aoff[entries] = static_cast<uint16_t>(R);
      }
    }
  }

  // The same for many rows, by one warp; ctl->cnt is zero on entry.
  static __device__ __forceinline__ void build_lists(const FewParams& p, Ctrl* ctl, int lane) {
    const int R = p.T * p.k;
    // a row's rank among the rows of its expert, 32 rows at a time
#pragma unroll 1
    for (int r0 = 0; r0 < R; r0 += 32) {
      const int r = r0 + lane, e = r < R ? ctl->ids[r] : -1 - lane;
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int before = r < R ? ctl->cnt[e] : 0;
      __syncwarp();
      if (r < R) {
        ctl->pos[r] = static_cast<uint16_t>(before + __popc(same & ((1u << lane) - 1u)));
        if ((same >> lane) == 1u) ctl->cnt[e] = before + __popc(same);  // the last of them
      }
      __syncwarp();
    }
    const int per = (p.E + 31) / 32;  // consecutive experts of a lane
    int rows = 0, act = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i, n = e < p.E ? ctl->cnt[e] : 0;
      rows += n;
      act += (n + kFewGroup - 1) / kFewGroup;
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
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i, n = e < p.E ? ctl->cnt[e] : 0;
      if (n > 0) ctl->amap[e] = static_cast<uint16_t>(ao);
      for (int i0 = 0; i0 < n; i0 += kFewGroup) {
        ctl->aexp[ao] = static_cast<uint16_t>(e);
        ctl->aoff[ao] = static_cast<uint16_t>(ro + i0);
        ++ao;
      }
      ro += n;
    }
    __syncwarp();
#pragma unroll 1
    for (int r = lane; r < R; r += 32) {
      const int at = ctl->aoff[ctl->amap[ctl->ids[r]]] + ctl->pos[r];
      ctl->srow[at] = static_cast<uint16_t>(r / p.k);
      ctl->pos[r] = static_cast<uint16_t>(at);
    }
    if (lane < p.T) ctl->srow[R + lane] = static_cast<uint16_t>(lane);
  }

  // The router's planes.  A unit is 64 experts x one slice of D x 8 NT tokens; its k16
  // steps go round the CTA's warps, two at a time.
  static __device__ __forceinline__ void router(const FewParams& p, float* red, int b, int G) {
    constexpr int NW = CT / 32, PL = Sm::kPlanes, PW = 8 * NT * 68;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, c = lane & 3;
    const int SE = (p.E + 63) / 64, steps = (p.D + 15) / 16;
    const bool vec = (p.E & 7) == 0;
#pragma unroll 1
    for (int u = b; u < SE * p.nplanes * ((p.T + 8 * NT - 1) / (8 * NT)); u += G) {
      const int se = u % SE, pl = u / SE % p.nplanes, t0 = u / (SE * p.nplanes) * 8 * NT;
      const int s0 = steps * pl / p.nplanes, s1 = steps * (pl + 1) / p.nplanes;
      float acc[NT][4][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[i][j][t] = 0.0f;
      const int col = se * 64 + g * 8;
#pragma unroll 1
      for (int st = s0 + wid; st < s1; st += 2 * NW) {
        uint32_t w[2][4][4], x[2][NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k0 = st + h * NW < s1 ? (st + h * NW) * 16 : p.D;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = k0 + 2 * c + (i & 1) + (i >> 1) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[h][i][j] = 0u;
            if (k < p.D) {
              const __nv_bfloat16* src = p.Wg + static_cast<size_t>(k) * p.E + col;
              if (vec) {
                if (col < p.E) {
                  const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
                  w[h][i][0] = v.x; w[h][i][1] = v.y; w[h][i][2] = v.z; w[h][i][3] = v.w;
                }
              } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (col + j < p.E)
                    w[h][i][j >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(src) + j))
                                       << (16 * (j & 1));
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int t = t0 + nt * 8 + g, k = k0 + 2 * c;
            x[h][nt][0] = x[h][nt][1] = 0u;
            if (t < p.T) {
              const __nv_bfloat16* src = p.x + static_cast<size_t>(t) * p.D + k;
              if (k < p.D) x[h][nt][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
              if (k + 8 < p.D) x[h][nt][1] = __ldg(reinterpret_cast<const uint32_t*>(src + 8));
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            const uint32_t a0 = __byte_perm(w[h][0][mt], w[h][1][mt], 0x5410);
            const uint32_t a1 = __byte_perm(w[h][0][mt], w[h][1][mt], 0x7632);
            const uint32_t a2 = __byte_perm(w[h][2][mt], w[h][3][mt], 0x5410);
            const uint32_t a3 = __byte_perm(w[h][2][mt], w[h][3][mt], 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816<false>(acc[nt][mt], a0, a1, a2, a3, x[h][nt][0], x[h][nt][1]);
          }
      }
      // warp w adds to plane w % PL in round w / PL
#pragma unroll 1
      for (int r = 0; r < NW / PL; ++r) {
        if (wid / PL == r) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              float* at = red + (wid % PL) * PW + (nt * 8 + 2 * c) * 68 + g * 8 + 2 * mt;
              const float* v = acc[nt][mt];
              if (r == 0) {
                at[0] = v[0]; at[68] = v[1]; at[1] = v[2]; at[69] = v[3];
              } else {
                at[0] += v[0]; at[68] += v[1]; at[1] += v[2]; at[69] += v[3];
              }
            }
        }
        bar();
      }
#pragma unroll 1
      for (int i = tid; i < min(8 * NT, p.T - t0) * 64; i += CT) {
        const int t = i >> 6, e = se * 64 + (i & 63);
        float v = red[t * 68 + (i & 63)];
#pragma unroll
        for (int q = 1; q < PL; ++q) v += red[q * PW + t * 68 + (i & 63)];
        if (e < p.E) p.planes[(static_cast<size_t>(pl) * p.T + t0 + t) * p.E + e] = v;
      }
      bar();
    }
  }

  // Token rows in the layout's k order, padded with zeros, a CTA for each (the
  // highest first: they have no router unit); fp16 rows by their power of two.
  static __device__ __forceinline__ void stage_x(const FewParams& p, float* red, int b, int G) {
    const int tid = threadIdx.x;
#pragma unroll 1
    for (int t = G - 1 - b; t < p.T; t += G) {
      const __nv_bfloat16* src = p.x + static_cast<size_t>(t) * p.D;
      uint16_t* dst = p.xp + static_cast<size_t>(t) * p.Dp;
      float sc = 1.0f;
      if constexpr (Tr::F16) {
        uint32_t m = 0;  // bf16 bits order as 16-bit whole numbers
        for (int k0 = tid * 8; k0 < p.D; k0 += CT * 8) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + k0));
          m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                   __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
        m = max(m & 0xffffu, m >> 16) << 16;
        m = __reduce_max_sync(0xffffffffu, m);
        uint32_t* all = reinterpret_cast<uint32_t*>(red);
        if ((tid & 31) == 0) all[tid >> 5] = m;
        bar();
        m = __reduce_max_sync(0xffffffffu, (tid & 31) < CT / 32 ? all[tid & 31] : 0u);
        bar();
        const int e = row_exp(m);
        sc = exp2_int(e);
        if (tid == 0) p.xinv[t] = exp2_int(-e);
      }
#pragma unroll 1
      for (int k0 = tid * 8; k0 < p.Dp; k0 += CT * 8) {
        union {
          uint4 v;
          __nv_bfloat16 h[8];
        } in;
        in.v = make_uint4(0, 0, 0, 0);
        if (k0 < p.D) in.v = __ldg(reinterpret_cast<const uint4*>(src + k0));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint16_t o;
          if constexpr (Tr::F16) o = __half_as_ushort(__float2half_rn(__bfloat162float(in.h[j]) * sc));
          else o = __bfloat16_as_ushort(in.h[j]);
          dst[perm_k<KIND, GRP>(k0 + j)] = o;
        }
      }
    }
  }
};

template <int KIND, int GRP, int NT>
__global__ void __launch_bounds__(FewSmem<KIND, GRP, NT>::kBlock, 1)
    few_layer_kernel(const __grid_constant__ CUtensorMap m13, const __grid_constant__ CUtensorMap m2,
                     const __grid_constant__ CUtensorMap m13s, const __grid_constant__ CUtensorMap m2s,
                     const __grid_constant__ FewParams p) {
  using F = Few<KIND, GRP, NT>;
  using Tr = StreamTraits<KIND, GRP>;
  using Sm = FewSmem<KIND, GRP, NT>;
  using Ctrl = typename Sm::Ctrl;
  constexpr int CT = Sm::kCons;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* red = reinterpret_cast<float*>(ring + Sm::NST * Sm::kSlot);
  Ctrl* ctl = reinterpret_cast<Ctrl*>(ring + Sm::NST * Sm::kSlot + Sm::kRedBufs * Sm::kRedBytes);
  StreamRing* sr = &ctl->ring;
  const int tid = threadIdx.x, b = blockIdx.x, G = gridDim.x, lane = tid & 31;
  const int R = p.T * p.k;
  const bool shared = p.Is > 0;

  if (tid == 0) sr->init(CT / 32);
  __syncthreads();

  if (tid >= CT + 32 + 32 * Sm::kFeeders) {  // ------------------------ finisher
    RedPos rpos;
    asm volatile("bar.sync 4, %0;" ::"n"(CT + 32 * Sm::kFeeders + 32) : "memory");  // the expert lists are built
    F::template finish<false>(p, ctl->pass[0], ctl, red, rpos, b, lane);
    asm volatile("bar.arrive 5, %0;" ::"n"(CT + 32) : "memory");  // h is written
    F::template finish<true>(p, ctl->pass[1], ctl, red, rpos, b, lane);
    asm volatile("bar.arrive 6, %0;" ::"n"(CT + 32) : "memory");  // y is written
    return;
  }
  if (tid >= CT + 32) {  // -------------------------------------------- feeders
    RingPos pos;
    const int me = (tid - CT - 32) >> 5;
    asm volatile("bar.sync 4, %0;" ::"n"(CT + 32 * Sm::kFeeders + 32) : "memory");  // x rows and expert lists are there
    bool ok = F::template feed<false>(p, ctl->pass[0], ctl, ring, pos, me, lane);
    asm volatile("bar.sync 3, %0;" ::"n"(CT + 32 * Sm::kFeeders) : "memory");  // h rows are there
    if (ok) ok = F::template feed<true>(p, ctl->pass[1], ctl, ring, pos, me, lane);
    if (!ok) sr->give_up(p.err);
    cp_async_wait_all();
    return;
  }
  if (tid >= CT) {  // ------------------------------------------------ producer
    if (lane == 0 && shared) {
      // in L2 beside what streams by: 32 MB of each projection
      F::template prefetch_shared<false>(p, &m13s, b, G, 2048 / G);
      F::template prefetch_shared<true>(p, &m2s, b, G, 2048 / G);
    }
    __syncwarp();
    asm volatile("bar.sync 2, %0;" ::"n"(CT + 32) : "memory");  // the expert lists are built
    if (lane == 0) {
      RingPos pos;
      const uint64_t policy = l2_policy_evict_first();
      bool ok = F::template produce<false>(&m13, &m13s, ctl->pass[0], ctl, sr, ring, pos, policy);
      if (ok) ok = F::template produce<true>(&m2, &m2s, ctl->pass[1], ctl, sr, ring, pos, policy);
      if (!ok) sr->give_up(p.err);
      if (sr->aborted()) drain_ring(sr, pos, Sm::NST);
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  // (every named barrier but the consumers' own is used once: a role without
  // work of its own may be at its next one before the others reach the last)
  if (tid == 0) p.cnt[b] = 0;
  // one token: k entries, whatever the routing
  if (p.T == 1 && tid >= 32 && tid < 34) ctl->pass[tid - 32] = few_pass<KIND, GRP>(p, tid == 33, p.k, G, b);
  if (Tr::F16)
    for (int r = b * CT + tid; r < R + p.T; r += G * CT) p.hmax[r] = 0;
  // phase 0 (no router weights: the experts are chosen already, in ids and topw)
  const bool given = p.Wg == nullptr;
  if (!given) F::router(p, red, b, G);
  F::stage_x(p, red, b, G);
  F::grid_sync(p, sr, 0, 3);

  // phase 1
  if (R > F::kPairRows)
    for (int e = tid; e < p.E; e += CT) ctl->cnt[e] = 0;
  if (!given && p.nplanes * p.T * p.E * 4 <= kFewPlaneBytes) {
    F::topk(p, 0, 1, b == 0, ctl->ids, ctl->w, red);
    if (b == 0)
      for (int r = tid; r < R; r += CT) {
        p.ids[r] = ctl->ids[r];
        p.topw[r] = ctl->w[r];
      }
  } else {
    if (!given) {
      F::topk(p, b, G, true, p.ids, p.topw, red);
      F::grid_sync(p, sr, 1, -1);
    }
    for (int r = tid; r < R; r += CT) {
      ctl->ids[r] = __ldcg(p.ids + r);
      ctl->w[r] = __ldcg(p.topw + r);
    }
    F::bar();
    // After a wait that gave up, or with arrivals left over from one, these may be any
    // numbers; the lists, and the room for an entry's rows, need k experts a token.
    bool bad = false;
    for (int r = tid; r < R; r += CT) {
      const int e = ctl->ids[r];
      bad |= static_cast<unsigned>(e) >= static_cast<unsigned>(p.E);
      for (int o = r - r % p.k; o < r; ++o) bad |= ctl->ids[o] == e;
    }
    if (bar_consumers_or<CT>(bad)) {
      for (int r = tid; r < R; r += CT) ctl->ids[r] = r % p.k;
      if (tid == 0) sr->give_up(p.err);
      F::bar();
    }
  }
  if (R <= F::kPairRows) F::build_lists_pairs(p, ctl, tid);
  if (tid < 32) {
    if (R > F::kPairRows) F::build_lists(p, ctl, lane);
    __syncwarp();
    if (p.T > 1 && lane < 2) ctl->pass[lane] = few_pass<KIND, GRP>(p, lane == 1, ctl->na, G, b);
  }
  F::bar();
  asm volatile("bar.arrive 4, %0;" ::"n"(CT + 32 * Sm::kFeeders + 32) : "memory");
  asm volatile("bar.arrive 2, %0;" ::"n"(CT + 32) : "memory");

  RingPos pos;
  RedPos rpos;
  const uint32_t ring_a = smem_u32(ring);
  // phase 2: gate/up
  F::template consume<false>(p, ctl->pass[0], ctl, ring_a, red, pos, rpos, b);
  asm volatile("bar.sync 5, %0;" ::"n"(CT + 32) : "memory");  // the finisher is through
  F::grid_sync(p, sr, 2, 0);
  asm volatile("bar.arrive 3, %0;" ::"n"(CT + 32 * Sm::kFeeders) : "memory");

  // phase 3: down
  const FewPass& dn = ctl->pass[1];
  // the h rows of the run's first strip into L1 at once: the feeders, which load
  // and convert them stage by stage, would wait for L2 at every stage
  if (Tr::F16) F::prefetch_h(p, dn, ctl);
  F::template consume<true>(p, dn, ctl, ring_a, red, pos, rpos, b);
  asm volatile("bar.sync 6, %0;" ::"n"(CT + 32) : "memory");  // the finisher is through
  F::grid_sync(p, sr, 3, 2);

  // phase 4: the weighted sum of a token's rows.  Eight columns a group of eight
  // lanes; lane l takes experts l, l + 8 and the shared expert as number k, and
  // the lanes' sums are added in a fixed tree.
  {
    const int per = p.D / 8, l = lane & 7, items = p.T * per;
    const int terms = p.k + (shared ? 1 : 0);
#pragma unroll 1
    // (item groups of a warp's four are dealt to the CTAs in turn)
    for (int w0 = (tid >> 5) * G + b; w0 * 4 < items; w0 += G * (CT / 32)) {
      const int i0 = w0 * 4 + (lane >> 3);
      const bool in = i0 < items;
      const int i = in ? i0 : items - 1;
      const int t = i / per, d0 = (i - t * per) * 8;
      const int s = d0 / (2 * Tr::HC), col = d0 % (2 * Tr::HC);
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = 0.0f;
      for (int j = l; j < terms; j += 8) {
        const bool rt = j < p.k;
        // the row, its place among the expert's rows, its entry and place there
        const int e = rt ? ctl->ids[t * p.k + j] : 0;
        const int r = rt ? ctl->pos[t * p.k + j] : R + t;
        const float4* src = reinterpret_cast<const float4*>(p.prim + static_cast<size_t>(r) * p.W +
                                                            static_cast<size_t>(s) * 2 * Tr::HC + col);
        const float4 y0 = __ldcg(src), y1 = __ldcg(src + 1);
        float w = rt ? ctl->w[t * p.k + j] : 1.0f;
        if constexpr (Tr::F16) w *= F::exp2_int(-F::row_exp(__ldcg(p.hmax + r)));
        float4 c0v = make_float4(1.0f, 1.0f, 1.0f, 1.0f), c1v = c0v;
        if constexpr (KIND == kStreamFp8 || KIND == kStreamFp8Nk) {
          const float4* sc = reinterpret_cast<const float4*>(
              static_cast<const float*>(rt ? p.s2 : p.s2s) + (rt ? static_cast<size_t>(e) * p.D : 0) + d0);
          c0v = __ldg(sc);
          c1v = __ldg(sc + 1);
        }
        float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
        const int at = rt ? r - ctl->aoff[ctl->amap[e]] : t;
        const int a = (rt ? ctl->amap[e] : 0) + at / kFewGroup, sl = at % kFewGroup;
        const int C = dn.C[rt];
        const long long q0 = (rt ? dn.shared : 0) + (static_cast<long long>(a) * dn.S[rt] + s) * C;
        const int c0 = few_cta(dn, q0), c1 = few_cta(dn, q0 + C - 1);
#pragma unroll 1
        for (int cta = c0 + 1; cta <= c1; ++cta) {
          const float4* x = reinterpret_cast<const float4*>(
              p.extra + (static_cast<size_t>(cta) * p.T + sl) * 2 * Tr::HC + col);
          const float4 m = __ldcg(x), n = __ldcg(x + 1);
          y[0] += m.x; y[1] += m.y; y[2] += m.z; y[3] += m.w;
          y[4] += n.x; y[5] += n.y; y[6] += n.z; y[7] += n.w;
        }
        const float cs[8] = {c0v.x, c0v.y, c0v.z, c0v.w, c1v.x, c1v.y, c1v.z, c1v.w};
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = fmaf(w, y[q] * cs[q], o[q]);
      }
#pragma unroll
      for (int m = 1; m < 8; m <<= 1)
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] += __shfl_xor_sync(0xffffffffu, o[q], m);
      if (in && l == 0) {
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
  if (sr->aborted()) drain_grace();  // copies that the producer could not wait for
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
    const uint32_t b13[4] = {Tr::QC, 1, Tr::BOX_ROWS, 1};
    const uint64_t d2[3] = {d, n, g}, t2[2] = {d * eb, n * d * eb};
    const uint32_t b2[3] = {Tr::QC, Tr::BOX_ROWS, 1};
    return encode_tmap(&m13, W13, 4, d13, t13, b13, dt) && encode_tmap(&m2, W2, 3, d2, t2, b2, dt);
  }
  const uint64_t kb = KIND == kStreamFp8Nk ? d : d / 2, nb = KIND == kStreamFp8Nk ? n : n / 2;
  const uint64_t d13[4] = {kb, n, 2, g}, t13[3] = {kb, n * kb, 2 * n * kb};
  const uint32_t b13[4] = {128, Tr::BOX_ROWS, 1, 1};
  const uint64_t d2[3] = {nb, d, g}, t2[2] = {nb, d * nb};
  const uint32_t b2[3] = {128, Tr::BOX_ROWS, 1};
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
  cfg.blockDim = dim3(Sm::kBlock);
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
  return launch_few_nt<KIND, GRP, 2>(a, s);
}

cudaError_t launch_few_bf16(const FewArgs& a, cudaStream_t s);
cudaError_t launch_few_fp8(const FewArgs& a, cudaStream_t s);
cudaError_t launch_few_fp8nk(const FewArgs& a, cudaStream_t s);
cudaError_t launch_few_w4(int group, const FewArgs& a, cudaStream_t s);

}  // namespace moe
