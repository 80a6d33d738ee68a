// The choice of experts of one token by one warp, by softmax or sigmoid scores with a
// bias, groups of experts, top-k and renormalised weights (moe_gate_t in moe.h).  Shared
// by the stand-alone kernel (gate.cu) and the router projection fused with it
// (router_sm103.cu), so that both take every decision the same way.
#pragma once

#include <cstdint>

#include "moe_internal.h"

namespace moe {

// A float's bits in an order that unsigned integers compare (-0 as +0).
__device__ __forceinline__ uint32_t ordered_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ float gate_sigmoid(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }

// (a, b) becomes the two largest of a >= b and c >= d.
__device__ __forceinline__ void merge_top2(float& a, float& b, float c, float d) {
  b = fmaxf(fminf(a, c), fmaxf(b, d));
  a = fmaxf(a, c);
}

// Lane l holds the token's projected logits of experts l EPL .. l EPL + EPL - 1 in v
// (E <= 32 EPL; entries past E are ignored), so that among lanes and within one the lower
// index comes first.  Writes the final logits to logits_row (when given), ids_row and
// w_row [k]; returns ids_row[lane] on lanes below k <= 32, -1 on the others.
//
// A group's value is found by lanes that hold whole parts of one group (the group's size a
// multiple of EPL, a power of two lanes: shuffles among them), else group after group.
template <int EPL>
__device__ __forceinline__ int warp_gate_topk(float (&v)[EPL], int lane, const GateParams& g,
                                              const float* __restrict__ logit_bias,
                                              const float* __restrict__ select_bias, float* logits_row,
                                              int32_t* __restrict__ ids_row, float* __restrict__ w_row,
                                              int32_t* err) {
  constexpr unsigned kFull = 0xffffffffu;
  const int e0 = lane * EPL, E = g.E, k = g.k;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    float x = -INFINITY;
    if (e0 + i < E) {
      x = v[i];
      if (logit_bias) x += logit_bias[e0 + i];
      if (logits_row) logits_row[e0 + i] = x;
      if (!isfinite(x)) {
        bad = true;
        x = -INFINITY;
      }
    }
    v[i] = x;
  }
  // softmax over all experts: its largest logit and the inverse of its sum, where the
  // scores themselves are needed (renormalised weights need only those chosen)
  const bool by_score = select_bias || (g.n_group > 1 && g.top2);
  float m = 0.0f, rz = 1.0f;
  if (!g.sigmoid && (by_score || !g.renorm)) {
    m = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (m == -INFINITY) m = 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) z += expf(v[i] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    rz = z > 0.0f ? 1.0f / z : 0.0f;
  }
  auto score = [&](float x) { return g.sigmoid ? gate_sigmoid(x) : expf(x - m) * rz; };
  float c[EPL];  // what is compared: the biased score, or the logit
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    c[i] = v[i];
    if (select_bias && e0 + i < E && v[i] != -INFINITY) {
      c[i] = score(v[i]) + select_bias[e0 + i];
      if (!isfinite(c[i])) {
        bad = true;
        c[i] = -INFINITY;
      }
    }
  }
  if (__any_sync(kFull, bad) && lane == 0) atomicOr(err, MOE_DEV_NONFINITE_LOGIT);

  uint32_t key[EPL];  // 0: not to be chosen (below every value's key, -infinity's too)
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = e0 + i < E ? ordered_key(c[i]) : 0u;

  if (g.topk_group < g.n_group) {
    const int size = E / g.n_group, lanes = size / EPL;
    // (of the two largest, b <= a; -infinity: not there)
    auto value = [&](float a, float b) {
      if (!g.top2 || a == -INFINITY) return a;
      if (select_bias) return b == -INFINITY ? a : a + b;
      return score(a) + score(b);
    };
    if (size % EPL == 0 && (lanes & (lanes - 1)) == 0) {
      float a = c[0], b = -INFINITY;
#pragma unroll
      for (int i = 1; i < EPL; ++i) merge_top2(a, b, c[i], -INFINITY);
      for (int o = 1; o < lanes; o <<= 1)
        merge_top2(a, b, __shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o));
      uint32_t gk = e0 < E ? ordered_key(value(a, b)) : 0u;
      bool kept = false;
      for (int j = 0; j < g.topk_group; ++j) {
        const uint32_t best = __reduce_max_sync(kFull, gk);
        const int first = __ffs(__ballot_sync(kFull, gk == best)) - 1;
        if (e0 < E && lane / lanes == first / lanes) {
          kept = true;
          gk = 0u;
        }
      }
      if (!kept) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = 0u;
      }
    } else {
      uint32_t gk = 0u;  // lane j: group j
      for (int j = 0; j < g.n_group; ++j) {
        float a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (e0 + i >= j * size && e0 + i < (j + 1) * size) merge_top2(a, b, c[i], -INFINITY);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          merge_top2(a, b, __shfl_xor_sync(kFull, a, o), __shfl_xor_sync(kFull, b, o));
        const uint32_t kj = ordered_key(value(a, b));
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
        if (e0 + i < E && !((kept >> ((e0 + i) / size)) & 1u)) key[i] = 0u;
    }
  }

  // k rounds: the largest key of the warp, the first lane that has it, its first entry
  float my_x = -INFINITY;  // logit of lane j's choice
  int my_e = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t bk = key[0];
    int bi = 0;
    float bx = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) {
      if (key[i] > bk) {
        bk = key[i];
        bi = i;
        bx = v[i];
      }
    }
    const uint32_t best = __reduce_max_sync(kFull, bk);
    const int from = __ffs(__ballot_sync(kFull, bk == best)) - 1;
    const float x = __shfl_sync(kFull, bx, from);
    const int e = from * EPL + __shfl_sync(kFull, bi, from);
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == bi) key[i] = 0u;
    }
    if (lane == j) {
      my_x = x;
      my_e = e;
    }
  }
  float top = my_x;  // largest chosen logit (lanes past k hold -infinity)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  float w;
  if (top == -INFINITY) {
    w = 1.0f / static_cast<float>(k);
  } else if (g.renorm) {
    // (e^l is sigmoid(l) in fp32 below -60, and more: it does not run out there)
    const float p = g.sigmoid && top > -60.0f ? gate_sigmoid(my_x) : expf(my_x - top);
    float z = lane < k ? p : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    w = p / z;
  } else {
    w = score(my_x);
  }
  if (lane >= k) return -1;
  ids_row[lane] = my_e;
  w_row[lane] = w * g.scale;
  return my_e;
}

}  // namespace moe
