"""64-bit reference of the few-token operators, with the error that the
kernels' arithmetic allows for each output element.

Unit roundoffs: fp32 sums are bounded with u32 = 2^-23 per addition (the tensor
core may truncate), so a sum of n products is off by at most n u32 times the
sum of the products' magnitudes; bf16 rounds by at most 2^-8 of the value.  With
bf16 weights h is carried as two bf16 terms, off by at most 2^-16 of the value;
with e4m3 and 4-bit weights x and h are fp16 rows times a power of two that puts
the row's largest element in [2^14, 2^15): h is off by at most 2^-11 of the
value, and an element that becomes subnormal there (x too) by at most half the
smallest step, 2^-25, that is 2^-39 of the row's largest.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -23
BF16 = 2.0 ** -8


def unpack_w4(q, s, zeros=None):
    """[.., N, K] fp64 values of 4-bit weights."""
    lo, hi = (q & 15).double(), (q >> 4).double()
    codes = torch.stack((lo, hi), -1).flatten(-2)
    g = codes.shape[-1] // s.shape[-1]
    z = 8.0 if zeros is None else (zeros & 15).double().repeat_interleave(g, -1)
    return (codes - z) * s.double().repeat_interleave(g, -1)


def dense(W, s, w_dtype):
    """[.., K, N] fp64 weights of any layout, scales included."""
    if w_dtype == "bf16":
        return W.double()
    if w_dtype == "fp8_e4m3":
        return W.double() * s.double()[..., None, :]
    if w_dtype == "fp8_e4m3_nk":
        return (W.double() * s.double()[..., :, None]).transpose(-1, -2)
    return unpack_w4(W, s).transpose(-1, -2)


def _ffn(x, W13, W2, act, fp16):
    """(y, allowed error of y) of one gated FFN, rows of x [n, D]."""
    D, I = W13.shape[0], W2.shape[0]
    gu, mag = x @ W13, x.abs() @ W13.abs()
    # a 4-bit or e4m3 scale multiplies a finished partial sum: two more roundings
    e = (D + 8) * U32 * mag
    if fp16:
        e = e + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * W13.abs().sum(0)
    g, u, eg, eu = gu[:, :I], gu[:, I:], e[:, :I], e[:, I:]
    if act == "swiglu":
        a = g / (1 + torch.exp(-g))
    else:
        a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    h = a * u
    # |act'| <= 1.13; the activation itself to 16 u32 of |g| (exp / tanh, a
    # division and a few products; tanh's absolute error counts against 1)
    eh = 1.13 * eg * u.abs() + (a.abs() + 1.13 * eg) * eu + 16 * U32 * g.abs() * u.abs()
    eh = eh + (2.0 ** -11 if fp16 else 2.0 ** -16) * (h.abs() + eh)
    if fp16:
        eh = eh + 2.0 ** -39 * (h.abs() + eh).amax(1, keepdim=True)
    y = h @ W2
    ey = eh @ W2.abs() + (I + 8) * U32 * ((h.abs() + eh) @ W2.abs())
    return y, ey


def layer(x, Wg, bias, W13, s13, W2, s2, W13s, s13s, W2s, s2s, w_dtype, k, act, renorm, ids):
    """(out, allowed error, exact logits, allowed error of a logit) on the CPU
    in fp64, for the experts `ids` [T, k] the kernel chose."""
    x = x.double()
    T, D = x.shape
    logits = x @ Wg.double() + (0.0 if bias is None else bias.double())
    el = (D + 20) * U32 * (x.abs() @ Wg.double().abs() + (0.0 if bias is None else bias.double().abs()))
    v = logits.gather(1, ids)
    top = v.amax(1, keepdim=True)
    w = torch.exp(v - top)
    w = w / (w.sum(1, keepdim=True) if renorm else torch.exp(logits - top).sum(1, keepdim=True))
    ew = w * (2 * el.amax(1, keepdim=True) + 64 * U32)
    out = torch.zeros_like(x)
    err = torch.zeros_like(x)
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        sc = (lambda s: None if s is None else s[e])
        y, ey = _ffn(x[t], dense(W13[e], sc(s13), w_dtype), dense(W2[e], sc(s2), w_dtype), act, w_dtype != "bf16")
        out.index_put_((t,), w[t, j, None] * y, accumulate=True)
        err.index_put_((t,), (w[t, j, None] + ew[t, j, None]) * ey + ew[t, j, None] * y.abs()
                       + (k + 2) * U32 * w[t, j, None] * y.abs(), accumulate=True)
    if W13s is not None:
        y, ey = _ffn(x, dense(W13s, s13s, w_dtype), dense(W2s, s2s, w_dtype), act, w_dtype != "bf16")
        out += y
        err += ey + 2 * U32 * (y.abs() + out.abs())
    return out, err + BF16 * (out.abs() + err), logits, el


def linear(x, q, s, zeros, out_dtype):
    """(y, allowed error) of x W^T."""
    W, x = unpack_w4(q, s, zeros), x.double()
    y, mag = x @ W.t(), x.abs() @ W.abs().t()
    e = (x.shape[1] + 8) * U32 * mag
    return y, e + (BF16 if out_dtype == torch.bfloat16 else 2.0 ** -24) * (y.abs() + e)
