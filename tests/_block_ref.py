"""64-bit references of the operators around the experts (moe_add_rms_norm,
moe_route_gated, moe_lora), with the error that the kernels' arithmetic allows.

A rounding is off by at most half a step, 2^-8 of the value for bf16 and 2^-24 for
fp32; e4m3 by 2^-4 of the value, or half its smallest step, 2^-10.  Sums on the
CUDA cores round to nearest (2^-24 an addition of what is added up), those of
mma.sync may truncate (2^-23).
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def norm(x, residual, weight, eps):
    """(s, y, allowed relative error of y before its rounding).  A thread adds up to 32
    squares, then come 5 + 5 steps of tree and at most 32 warps in turn: 74 roundings of
    the sum, halved by the root; the root's two ulps; s, the product with the root, with the
    weight."""
    s = x.double() + (0.0 if residual is None else residual.double())
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * weight.double()
    return s, y, (74 / 2 + 4 + 2 + 3) * U


def rounded(v, dtype, rel):
    """Allowed error of v computed to `rel` and rounded to `dtype` (the last term: where the
    type's values become subnormal)."""
    return v.abs() * (rel + HALF[dtype] * (1 + rel)) + 2.0 ** -133


def e4m3(y, group, rel):
    """(scales, allowed error of q times its scale, both for y computed to `rel`)."""
    T, D = y.shape
    s = y.view(T, -1, group or D).abs().amax(2) / 448
    s = torch.where(s > 0, s.clamp(min=2.0 ** -126), torch.ones_like(s))
    wide = s.repeat_interleave(group or D, dim=1)
    more = 2 * rel + 8 * U  # y, the scale, its inverse, their product
    return s, wide, torch.maximum(y.abs() * 2.0 ** -4, wide * 2.0 ** -10) * (1 + more) + 2 * more * y.abs()


def gate(logits, select_bias, k, score="sigmoid", n_group=1, topk_group=1, group_score="top2_sum", scale=1.0,
         renorm=True):
    """(ids, weights, margin) of rows of logits, token by token in plain Python: margin is
    the smallest difference, exact ties apart, that a choice or an order hangs on."""
    ids, w, margin = [], [], math.inf
    bias = None if select_bias is None else select_bias.double().tolist()
    for row in logits.double().tolist():
        E = len(row)
        l = [v if math.isfinite(v) else -math.inf for v in row]
        if score == "sigmoid":
            p = [math.exp(v) if v < -700 else 1 / (1 + math.exp(-v)) for v in l]
        else:
            m = max(l)
            z = [0.0 if v == -math.inf else math.exp(v - m) for v in l]
            p = [v / (sum(z) or 1.0) for v in z]
        c = [-math.inf if l[e] == -math.inf else p[e] + (bias[e] if bias else 0.0) for e in range(E)]
        c = [v if math.isfinite(v) else -math.inf for v in c]
        size = E // n_group

        def order(v, n):
            nonlocal margin
            got = sorted(range(len(v)), key=lambda i: (-v[i], i))
            for a, b in zip(got[:n], got[1:n + 1]):
                if v[a] != v[b] and v[b] != -math.inf:
                    margin = min(margin, v[a] - v[b])
            return got[:n]

        kept = list(range(E))
        if topk_group < n_group:
            vals = []
            for g in range(n_group):
                top = sorted(c[g * size:(g + 1) * size], reverse=True)
                two = [v for v in top[:2] if v != -math.inf] if group_score == "top2_sum" else top[:1]
                vals.append(sum(two) if two else -math.inf)
            groups = order(vals, topk_group)
            kept = sorted(e for g in groups for e in range(g * size, (g + 1) * size))
        chosen = [kept[i] for i in order([c[e] for e in kept], k)]
        q = [p[e] for e in chosen]
        if all(l[e] == -math.inf for e in chosen):
            q = [1 / k] * k
        elif renorm:
            if score == "softmax" or max(l[e] for e in chosen) < -700:
                m = max(l[e] for e in chosen)
                q = [0.0 if l[e] == -math.inf else math.exp(l[e] - m) for e in chosen]
            q = [v / sum(q) for v in q]
        ids.append(chosen)
        w.append([v * scale for v in q])
    return torch.tensor(ids), torch.tensor(w, dtype=torch.float64), margin


def lora(x, ids, A, B, scales, base, y_dtype):
    """(y, allowed error).  The sums over K and r truncate at most; x A^T times its scale is
    carried in two bf16 terms (2^-16) for bf16 y, three (2^-24) for fp32."""
    n, r, K = A.shape
    T, N = x.shape[0], B.shape[1]
    y = torch.zeros((T, N), dtype=torch.float64, device=x.device) if base is None else base.double().clone()
    err = torch.zeros_like(y)
    terms = 2.0 ** -16 if y_dtype == torch.bfloat16 else 2.0 ** -24
    for a in ids.unique().tolist():
        if not 0 <= a < n:
            continue
        t = (ids == a).nonzero()[:, 0]
        xa, Aa, Ba = x[t].double(), A[a].double(), B[a].double()
        s = 1.0 if scales is None else float(scales[a])
        v = s * (xa @ Aa.t())
        ev = abs(s) * (K + 80) * 2 * U * (xa.abs() @ Aa.abs().t())
        ev = ev + terms * (v.abs() + ev)
        d, mag = v @ Ba.t(), (v.abs() + ev) @ Ba.abs().t()
        y[t] += d
        err[t] += ev @ Ba.abs().t() + (3 * r + 8) * 2 * U * mag + 2 * U * (y[t].abs() + mag)
    return y, err + HALF[y_dtype] * (y.abs() + err) + 2.0 ** -133
