// The choice of experts of one token by one warp, by softmax or sigmoid scores with a
// bias, groups of experts, top-k and renormalised weights (moe_gate_t in moe.h).  Shared
// by the stand-alone kernel (gate.cu) and the router projection fused with it
// (router_sm103.cu), so that both take every decision the same way.
#pragma once

#include <cstdint>

#include "moe_internal.h"

namespace moe {

// A float's bits in an order that unsigned integers compare (-0 below +0).
__device__ __forceinline__ uint32_t ordered_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// e^x by the hardware's 2^x: off by 2^-22 and 2^-23 |x| of the value at most (of a sigmoid by
// half an ulp of 1), for what is compared; weights take expf and the quotients below.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
// a / b for b of 2^-100 to 2^100, |a| <= b: the product with the hardware's inverse, within
// three ulps, corrected by its remainder, which leaves half an ulp and 2^-20 of one (the rounding
// division's own code takes 0.3 us a call and 1.3 us for 16384 tokens).
__device__ __forceinline__ float gate_quotient(float a, float b) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}
template <bool FAST>
__device__ __forceinline__ float gate_sigmoid(float x) {
  float r;
  if (FAST) {
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + fast_exp(-x)));
    return r;
  }
  const float d = 1.0f + expf(-x);  // 1 to infinity: as gate_quotient, down to subnormal results
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
  return d < INFINITY ? fmaf(fmaf(-d, r, 1.0f), r, r) : 0.0f;
}

// (a, b) becomes the two largest of a >= b and c >= d.
__device__ __forceinline__ void merge_top2(uint32_t& a, uint32_t& b, uint32_t c, uint32_t d) {
  b = max(min(a, c), max(b, d));
  a = max(a, c);
}

// Descending (Batcher's odd-even merge sort: 19 exchanges for 8, 63 for 16).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&s)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t x = s[i + j], y = s[i + j + q];
            s[i + j] = max(x, y);
            s[i + j + q] = min(x, y);
          }
}

template <int EPL>
__device__ __forceinline__ void put_lane(uint32_t* to, const uint32_t (&s)[EPL]) {
  if constexpr (EPL == 2) {
    *reinterpret_cast<uint2*>(to) = make_uint2(s[0], s[1]);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) *reinterpret_cast<uint4*>(to + i) = make_uint4(s[i], s[i + 1], s[i + 2], s[i + 3]);
  }
}

// (a lane's keys and a 0 behind them, rows of 16 bytes)
__host__ __device__ constexpr int gate_scratch(int epl) { return 32 * ((epl + 4) / 4 * 4); }

// Lane l holds the token's projected logits of experts l EPL .. l EPL + EPL - 1 in v
// (E <= 32 EPL; entries past E are ignored, but are numbers), so that among lanes and within
// one the lower index comes first.  Writes the final logits to logits_row (when given), ids_row and
// w_row [k]; returns ids_row[lane] on lanes below k <= 16, -1 on the others.
//   WHOLE    E is a multiple of EPL: a lane has all its entries or none.
//   SIGMOID, BIAS  as g.sigmoid and select_bias say (no branch an entry on them).
//   scratch  gate_scratch(EPL) words of the warp's own in shared memory, 16-byte aligned.
//
// Bound by instructions, most of them on the half-rate integer pipe, so each lane sorts
// its keys once and the k rounds look at one head a lane: a warp maximum, the first lane
// that has it, and that lane's next key from shared memory.  Which entry of the lane a
// chosen key is, is found once at the end, by k lanes at a time.  A group's value comes from
// the sorted keys of the lanes that hold it (the group's size a multiple of EPL, a power of
// two lanes), else group after group.  Measured (one GB300, from a graph): 16384 tokens of 256
// experts in 8 groups, 4 kept, top-8, sigmoid and bias 12.3 us (656 instructions a token, which
// are 8.5 us at one a cycle on each scheduler; reading the logits would take 2.6; every round over
// all keys 28.0), 509 tokens of 512 experts, top-10, softmax and bias 3.7 us, one token 2.4 us.
template <int EPL, bool WHOLE, bool SIGMOID, bool BIAS>
__device__ __forceinline__ int warp_gate_topk(float (&v)[EPL], int lane, const GateParams& g,
                                              const float* __restrict__ logit_bias,
                                              const float* __restrict__ select_bias, float* logits_row,
                                              int32_t* __restrict__ ids_row, float* __restrict__ w_row,
                                              uint32_t* scratch, int32_t* err) {
  const bool bias_vec = !(reinterpret_cast<uintptr_t>(select_bias) & 15);
  constexpr unsigned kFull = 0xffffffffu;
  const int e0 = lane * EPL, E = g.E, k = g.k;
  const bool here = e0 < E;
  auto has = [&](int i) { return WHOLE || e0 + i < E; };  // (of a lane that is here)
  constexpr int kRow = gate_scratch(EPL) / 32;
  uint32_t* mine = scratch + lane * kRow;
  bool bad = false;
  {
    float zero = 0.0f;  // NaN once an entry is not finite
    if (logit_bias && here) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (has(i)) v[i] += logit_bias[e0 + i];
    }
    if (logits_row && here) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (has(i)) logits_row[e0 + i] = v[i];
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      zero = fmaf(v[i], 0.0f, zero);
      if (!has(i)) v[i] = -INFINITY;
    }
    if (!(zero == 0.0f)) {
      bad = true;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!isfinite(v[i])) v[i] = -INFINITY;
    }
  }
  const bool grouped = g.topk_group < g.n_group;
  // softmax over all experts: its largest logit and the inverse of its sum, where the
  // scores themselves are needed (renormalised weights need only those chosen)
  const bool scores = BIAS || (grouped && g.top2) || !g.renorm;
  float m = 0.0f, rz = 1.0f;
  if (!SIGMOID && scores) {
    m = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
    m = ordered_value(__reduce_max_sync(kFull, here ? ordered_key(m) : 0x007fffffu));  // (-infinity's)
    if (m == -INFINITY) m = 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) z += expf(v[i] - m);
    if (!here) z = 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    rz = z > 0.0f ? 1.0f / z : 0.0f;
  }
  auto score = [&](float x) { return SIGMOID ? gate_sigmoid<false>(x) : expf(x - m) * rz; };
  auto compared = [&](float x) { return SIGMOID ? gate_sigmoid<true>(x) : fast_exp(x - m) * rz; };
  // keys of what is compared, the biased score or the logit; 0: not to be chosen (below
  // every value's key, -infinity's too)
  uint32_t key[EPL];
  if (BIAS) {
    float c[EPL], zero = 0.0f;
    if (WHOLE && EPL % 4 == 0 && bias_vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        const float4 f = here ? *reinterpret_cast<const float4*>(select_bias + e0 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        c[i] = f.x, c[i + 1] = f.y, c[i + 2] = f.z, c[i + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = here && has(i) ? select_bias[e0 + i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      c[i] += compared(v[i]);
      zero = fmaf(c[i], 0.0f, zero);
    }
    // (a lane past E compares no expert's: 0 against a largest logit far below it is infinite)
    if (here && (bad || !(zero == 0.0f))) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const bool out = !isfinite(c[i]);  // (its weight, which is taken from v, is 0 too)
        bad |= out;
        if (out) v[i] = -INFINITY;
        if (v[i] == -INFINITY) c[i] = -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = has(i) ? ordered_key(c[i]) : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = has(i) ? ordered_key(v[i] + 0.0f) : 0u;  // (-0 as +0)
  }
  if (__any_sync(kFull, bad) && lane == 0) atomicOr(err, MOE_DEV_NONFINITE_LOGIT);

  // a group's value as a key, of the keys a >= b of its two largest
  auto group_key = [&](uint32_t ka, uint32_t kb) {
    const float a = ordered_value(ka), b = ordered_value(kb);
    if (!g.top2 || a == -INFINITY) return ka;
    const bool two = kb != 0u && b != -INFINITY;
    if (BIAS) return ordered_key(two ? a + b : a);
    return ordered_key(compared(a) + (two ? compared(b) : 0.0f));
  };
  const int size = grouped ? E / g.n_group : E, lanes = size / EPL;
  const bool by_lanes = size % EPL == 0 && (lanes & (lanes - 1)) == 0;
  if (grouped && !by_lanes) {
    uint32_t gk = 0u;  // lane j: group j
    for (int j = 0; j < g.n_group; ++j) {
      uint32_t a = 0u, b = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (e0 + i >= j * size && e0 + i < (j + 1) * size) merge_top2(a, b, key[i], 0u);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        merge_top2(a, b, __shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o));
      const uint32_t kj = group_key(a, b);
      if (lane == j) gk = kj;
    }
    uint32_t kept = 0u;
    for (int j = 0; j < g.topk_group; ++j) {
      const uint32_t best = __reduce_max_sync(kFull, gk);
      const int first = __ffs(__ballot_sync(kFull, gk == best)) - 1;
      kept |= 1u << first;
      if (lane == first) gk = 0u;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (here && has(i) && !((kept >> ((e0 + i) / size)) & 1u)) key[i] = 0u;
  }
  uint32_t s[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) s[i] = key[i];
  sort_keys(s);
  uint32_t head = here ? s[0] : 0u;
  if (grouped && by_lanes) {
    uint32_t a = s[0], b = s[1];
    for (int o = 1; o < lanes; o <<= 1)
      merge_top2(a, b, __shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o));
    uint32_t gk = here ? group_key(a, b) : 0u;
    const int shift = 31 - __clz(lanes);
    bool kept = false;
    for (int j = 0; j < g.topk_group; ++j) {
      const uint32_t best = __reduce_max_sync(kFull, gk);
      const int first = __ffs(__ballot_sync(kFull, gk == best)) - 1;
      if (here && lane >> shift == first >> shift) {
        kept = true;
        gk = 0u;
      }
    }
    if (!kept) head = 0u;  // (its other keys are then never looked at)
  }

  __syncwarp();
  put_lane(mine, s);
  mine[EPL] = 0u;
  int my_from = 0;
  const uint32_t* next = mine;
  uint32_t my_key = 0u;
  for (int j = 0; j < k; ++j) {
    const uint32_t best = __reduce_max_sync(kFull, head);
    const int from = __ffs(__ballot_sync(kFull, head == best)) - 1;
    if (lane == from) head = *++next;
    if (lane == j) {
      my_key = best;
      my_from = from;
    }
  }
  // the entry of lane my_from: the first with this key, or, where the lane gave the same key
  // in the rounds just before (equal keys are chosen one after another), the one after those
  __syncwarp();
  put_lane(mine, key);
  __syncwarp();
  const uint32_t* theirs = scratch + my_from * kRow;
  const uint32_t up_key = __shfl_up_sync(kFull, my_key, 1);
  const int up_from = __shfl_up_sync(kFull, my_from, 1);
  const uint32_t again = __ballot_sync(kFull, lane > 0 && lane < k && my_key == up_key && my_from == up_from);
  int idx = 0;
  if (again == 0u) {
#pragma unroll
    for (int i = EPL - 1; i > 0; --i)
      if (theirs[i] == my_key) idx = i;
    if (theirs[0] == my_key) idx = 0;
  } else {
    int skip = lane - (31 - __clz(~again & ((2u << lane) - 1u)));
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (theirs[i] == my_key && skip-- == 0) idx = i;
  }
  float my_x = ordered_value(my_key);  // logit of lane j's choice
  if (BIAS) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = __float_as_uint(v[i]);
    put_lane(mine, key);
    __syncwarp();
    my_x = __uint_as_float(theirs[idx]);
  }
  if (lane >= k) my_x = -INFINITY;

  float w;
  if (!g.renorm && __shfl_sync(kFull, my_x, 0) != -INFINITY) {
    w = score(my_x);
  } else {
    // (a softmax's first choice, where its scores were not needed, is its largest logit)
    const float first = __shfl_sync(kFull, my_x, 0);
    float p = SIGMOID || scores ? score(my_x) : expf(my_x - (first == -INFINITY ? 0.0f : first));
    if (lane >= k) p = 0.0f;
    float z = p;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    if (__shfl_sync(kFull, z, 0) > 1e-25f) {
      w = gate_quotient(p, z);
    } else {
      // scores that run out of range: of a softmax, those beside its largest; sigmoids, which
      // are e^l there.  Their ratios are the exponentials of differences
      float top = my_x;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      p = lane >= k ? 0.0f : top == -INFINITY ? 1.0f : expf(my_x - top);
      z = p;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
      w = gate_quotient(p, z);
    }
  }
  if (lane >= k) return -1;
  const int e = my_from * EPL + idx;
  ids_row[lane] = e;
  w_row[lane] = w * g.scale;
  return e;
}

}  // namespace moe
