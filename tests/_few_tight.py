"""How far moe_layer_few may be from 64 bits, from the size of its sums' errors
rather than from their number times the sum of all magnitudes: for long sums, where
the latter allows more than the result itself.

For a sum of n products a_i b_i of either sign let s = sqrt(sum a_i^2 b_i^2), the
size that it has.

* fp32 sums: an accumulation is off by at most 2^-23 of the running sum (the tensor
  core may truncate), and a running sum stays below 6 s but for 1 in 10^8.  The
  accumulations of a sum of n products are at most n / 8 + 64 (n / 16 steps of the
  tensor core; with group scales one more for every 32; warps, teams, CTAs): the error
  is at most c(n) s, c(n) = 6 (n / 8 + 64) 2^-23.
* h is rounded, at most 2^-11 (fp16 rows) or 2^-16 (two bf16 terms) of the value, and
  carries the error of its own sums.  These errors differ from h to h in size and sign:
  an output that adds up errors of at most d_k W_kn is off by more than t times
  sqrt(sum d_k^2 W_kn^2) with a probability below 2 exp(-t^2 / 2) (Hoeffding): t = 8 for
  a single output, and 1 for the root mean square of all of them.  What truncation does
  to all of them alike, a part of at most 2 (D / 8 + 64) 2^-23, is allowed for beside it.
* The output is rounded to bf16, at most 2^-8 of the value; as the roundings lie evenly
  in their steps, their root mean square is at most 2^-8 / sqrt(3) of that of the
  values, and 1.05 of it over some thousand outputs.
"""
from __future__ import annotations

import math

import torch

from tests._few_ref import BF16, U32, dense


def _c(n: int) -> float:
    return 6 * (n / 8 + 64) * U32


def _ffn(x, W13, W2, act, fp16):
    """(y, error that is allowed as it is, sum of squares of those that add up at random)"""
    D, I = W13.shape[0], W2.shape[0]
    gu = x @ W13
    e = _c(D) * (x.square() @ W13.square()).sqrt() + 8 * U32 * gu.abs()
    if fp16:  # elements of x that become subnormal
        e = e + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * W13.abs().sum(0)
    g, u, eg, eu = gu[:, :I], gu[:, I:], e[:, :I], e[:, I:]
    if act == "swiglu":
        a = g / (1 + torch.exp(-g))
    else:
        a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    h = a * u
    # |act'| <= 1.13, the activation itself to 16 roundings of |g|
    eh = 1.13 * eg * u.abs() + (a.abs() + 1.13 * eg) * eu + 16 * U32 * g.abs() * u.abs()
    eh = eh + (2.0 ** -11 if fp16 else 2.0 ** -16) * h.abs()
    if fp16:
        eh = eh + 2.0 ** -39 * h.abs().amax(1, keepdim=True)
    y = h @ W2
    W2s = W2.square()
    return y, _c(I) * (h.square() @ W2s).sqrt() + (2 * (D / 8 + 64) + 8) * U32 * y.abs(), eh.square() @ W2s


def layer(x, Wg, bias, W13, s13, W2, s2, W13s, s13s, W2s, s2s, w_dtype, k, act, renorm, ids):
    """(out, error allowed as it is, sum of squares) in 64 bits for the experts `ids`."""
    x, Wg = x.double(), Wg.double()
    logits = x @ Wg + (0.0 if bias is None else bias.double())
    el = _c(x.shape[1]) * (x.square() @ Wg.square()).sqrt() + 8 * U32 * logits.abs()
    v = logits.gather(1, ids)
    top = v.amax(1, keepdim=True)
    w = torch.exp(v - top)
    w = w / (w.sum(1, keepdim=True) if renorm else torch.exp(logits - top).sum(1, keepdim=True))
    ew = w * (2 * el.amax(1, keepdim=True) + 64 * U32)
    fp16 = w_dtype != "bf16"
    out, lin, var = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        sc = (lambda s: None if s is None else s[e])
        y, ey, vy = _ffn(x[t], dense(W13[e], sc(s13), w_dtype), dense(W2[e], sc(s2), w_dtype), act, fp16)
        p, ep = w[t, j, None], ew[t, j, None]
        out.index_put_((t,), p * y, accumulate=True)
        lin.index_put_((t,), (p + ep) * ey + ep * y.abs() + (k + 2) * U32 * p * y.abs(), accumulate=True)
        var.index_put_((t,), (p + ep).square() * vy, accumulate=True)
    if W13s is not None:
        y, ey, vy = _ffn(x, dense(W13s, s13s, w_dtype), dense(W2s, s2s, w_dtype), act, fp16)
        out += y
        lin += ey + 2 * U32 * (y.abs() + out.abs())
        var += vy
    return out, lin, var


def verdict(out, want, lin, var):
    """(largest error over the allowed one, root mean square over the allowed one) of
    bf16 outputs; both at most 1 where the outputs are right."""
    err = (out.double() - want).abs()
    one = lin + 8 * var.sqrt()
    worst = (err / (one + BF16 * (want.abs() + one))).max().item()
    rms = (lambda v: v.square().mean().sqrt().item())
    return worst, rms(err) / (1.05 * BF16 / math.sqrt(3) * rms(want) + rms(lin) + rms(var.sqrt()))
