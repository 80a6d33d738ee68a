"""The bound of _few_tight, on the CPU at the widths of the GPU tests that use it
(with fewer experts): results in the kernels' arithmetic pass, mistakes of one step
of a long sum, one stage, one expert or one token do not."""
import pytest
import torch

from tests import _few_tight as tight
from tests._few_ref import dense

SHAPES = [
    # T, D, E, k, I, Is, w_dtype
    (12, 8192, 4, 2, 128, 4096, "w4_g64"),
    (12, 4096, 4, 2, 128, 2048, "bf16"),
    (3, 8192, 2, 2, 2048, 64, "w4_g32"),
    (1, 8192, 8, 8, 576, 0, "w4_g32"),
    (32, 1024, 4, 4, 1024, 0, "fp8_e4m3_nk"),
]


def _quantise(W, w):
    """[.., K, N] -> weights and scales in the layout of `w`."""
    if w == "bf16":
        return W.bfloat16(), None
    if w.startswith("fp8"):
        s = W.abs().amax(-2) / 448
        q = (W / s.unsqueeze(-2)).clamp(-448, 448).to(torch.float8_e4m3fn)
        return (q.transpose(-1, -2).contiguous() if w.endswith("nk") else q), s
    g = int(w[4:])
    Wt = W.transpose(-1, -2).contiguous().unflatten(-1, (-1, g))
    s = (Wt.abs().amax(-1) / 7).bfloat16()
    c = ((Wt / s.float()[..., None]).round().clamp(-8, 7) + 8).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _inputs(T, D, E, k, I, Is, w):
    g = torch.Generator().manual_seed(T + D)
    n = (lambda *s, std=1.0: torch.empty(s).normal_(0, std, generator=g))
    d = {"x": n(T, D).bfloat16(), "Wg": n(D, E, std=0.05).bfloat16(), "bias": None}
    d["W13"], d["s13"] = _quantise(n(E, D, 2 * I, std=0.05), w)
    d["W2"], d["s2"] = _quantise(n(E, I, D, std=0.05), w)
    d["W13s"], d["s13s"] = _quantise(n(D, 2 * Is, std=0.05), w) if Is else (None, None)
    d["W2s"], d["s2s"] = _quantise(n(Is, D, std=0.05), w) if Is else (None, None)
    return d


def _fp16_rows(h):
    s = 2.0 ** (14 - torch.floor(torch.log2(h.abs().amax(1, keepdim=True))))
    return (h * s).half().float() / s


def _run(d, w, ids, k, mistake=""):
    """The layer in fp32 sums and the kernels' roundings of h, with a mistake in it."""
    x, D = d["x"].float(), d["x"].shape[1]
    logits = d["x"].double() @ d["Wg"].double()
    p = torch.softmax(logits.gather(1, ids), 1).float()
    sc = (lambda s, e: None if s is None else s[e])
    if "flat" not in d:  # fp32 weights, once
        d["flat"] = [(dense(a, sa, w).float(), dense(b, sb, w).float()) for a, sa, b, sb in
                     [*((d["W13"][e], sc(d["s13"], e), d["W2"][e], sc(d["s2"], e)) for e in range(len(d["W13"])))] +
                     ([(d["W13s"], d["s13s"], d["W2s"], d["s2s"])] if d["W13s"] is not None else [])]

    def ffn(x, e, mistake):
        W13, W2 = d["flat"][e]
        if mistake in ("step", "down", "stage"):
            W13, W2 = W13.clone(), W2.clone()
        if mistake == "step":  # 16 inputs of 64 columns of gate and of up
            I = W2.shape[0]
            W13[D // 2:D // 2 + 16, :64] = 0
            W13[D // 2:D // 2 + 16, I:I + 64] = 0
        if mistake == "down":  # 16 of the down product's inputs, in 128 columns
            W2[16:32, 128:256] = 0
        if mistake == "stage":
            W13[:256] = 0
        gu = x @ W13
        I = W2.shape[0]
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        if w == "bf16":
            hi = h.bfloat16().float()
            h = hi + (h - hi).bfloat16().float()
        else:
            h = _fp16_rows(h)
        return h @ W2

    out = torch.zeros_like(x)
    last = ids.unique().tolist()[-1]
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        if mistake == "routed" or (mistake == "expert" and e == last):
            continue
        y = ffn(x[t], e, mistake if e == last else "")
        if mistake == "token" and e == last:  # another token's row
            y = y.clone()
            y[0] = ffn(x[(t[:1] + 1) % len(x)] if len(x) > 1 else x.flip(1), e, "")[0]
        out.index_put_((t,), p[t, j, None] * y, accumulate=True)
    if d["W13s"] is not None and mistake != "shared":
        out += ffn(x, -1, "")
    if mistake == "element":
        out[0, 5] = out[0, 6]
    if mistake == "zeros":
        out.zero_()
    return out.bfloat16()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_bound_tells_right_from_wrong(shape):
    T, D, E, k, I, Is, w = shape
    d = _inputs(*shape)
    logits = d["x"].double() @ d["Wg"].double()
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    want, lin, var = tight.layer(d["x"], d["Wg"], None, d["W13"], d["s13"], d["W2"], d["s2"], d["W13s"], d["s13s"],
                                 d["W2s"], d["s2s"], w, k, "swiglu", True, ids)
    worst, rms = tight.verdict(_run(d, w, ids, k), want, lin, var)
    assert worst <= 1 and rms <= 1
    mistakes = ["step", "down", "stage", "routed", "expert", "token", "element", "zeros"] + (["shared"] if Is else [])
    for m in mistakes:
        worst, rms = tight.verdict(_run(d, w, ids, k, m), want, lin, var)
        assert worst > 1 or rms > 1, f"{m}: {worst}, {rms}"
