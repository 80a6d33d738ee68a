"""moe_add_rms_norm, moe_route_gated and moe_lora on the GPU, where their inputs
or sizes are at an end of what they take."""
import math

import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests import _block_ref as ref
from tests._lib import ensure_library
from tests.test_gpu_block import BF16, F32, W_REL, WD, _block, _block_inputs, _gate, _gen, _normal, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


# ------------------------------------------------------------------- norm
def _codes(x, res, w, eps, group):
    """(y, q, scales) of moe_add_rms_norm; y of fp32 inputs is what q is made of."""
    T, D = x.shape
    y, q = torch.empty_like(x), torch.empty((T, D), dtype=torch.uint8, device="cuda")
    s = torch.empty((T, D // (group or D)), device="cuda")
    moe.moe_add_rms_norm(T, D, x, res, w, eps, None, y, q, s, group)
    return y, q, s


def _divided(y, s, group):
    """e4m3 codes of y / scale by fp32 division and torch's conversion, nearest even (on the host)."""
    v = y.cpu().view(y.shape[0], -1, group or y.shape[1]) / s.cpu()[:, :, None]
    return v.view_as(y).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("T,D,group", [(300, 4096, 0), (300, 4096, 32), (1000, 2816, 128), (400, 8192, 64), (700, 8192, 0), (200, 20480, 0), (200, 20480, 128)])
def test_norm_codes_are_those_of_the_quotients(T, D, group):
    """q = e4m3(y / scale): no code next to it where the quotient lies near the middle of two."""
    g = _gen(T + D + group)
    x, res = _normal((T, D), 1, g), _normal((T, D), 2, g)
    w = (1 + _normal((D,), 0.2, g, F32)).to(BF16)
    x[0], res[0, 1::2] = 0, 0  # zeros, of either sign
    x[0, 3], res[0, 3] = -0.0, -0.0
    y, q, s = _codes(x.float(), res.float(), w.float(), 1e-6, group)
    most = y.cpu().abs().view(T, -1, group or D).amax(2)
    assert torch.equal(s.cpu(), torch.where(most > 0, most / 448, torch.ones_like(most)))
    assert torch.equal(q.cpu(), _divided(y, s, group))
    _, q16, s16 = _codes(x, res, w, 1e-6, group)  # the same values in bf16: the same rows
    assert torch.equal(q16, q) and torch.equal(s16, s)


@pytest.mark.parametrize("e", [-124, -119, -110, -80, -64, -62, -60, -40, 60, 100, 120, 125])
def test_norm_codes_at_the_ends_of_the_range(e):
    """Scales near the smallest normal number and the largest; the smallest is 2^-126."""
    T, D = 64, 4096
    g = _gen(e + 200)
    x = _normal((T, D), 1, g, F32)
    w = torch.full((D,), 2.0 ** e, device="cuda")
    for group in (0, 128):
        y, q, s = _codes(x, None, w, 0.0, group)
        assert bool(y.isfinite().all())
        most = y.cpu().abs().view(T, -1, group or D).amax(2)
        assert torch.equal(s.cpu(), (most / 448).clamp(min=2.0 ** -126))
        assert torch.equal(q.cpu(), _divided(y, s, group))


# ------------------------------------------------------------------- gate
def _far_logits(E):
    """Rows whose largest logit is far below 0: finite, the type's lowest value among them."""
    low = torch.finfo(F32).min
    rows = torch.full((6, E), -100.0)
    rows[1, E // 2:] = low
    rows[2, :] = low
    rows[3] = -torch.linspace(89, 2000, E)
    rows[4, 1:] = low
    rows[5] = -60.0
    return rows


def _softmax_choice(logits, sb, k):
    """ids and renormalised weights of softmax scores with a bias, in 64 bits."""
    p = torch.softmax(logits.double(), dim=1)
    ids = torch.sort(p + sb.double(), dim=1, descending=True, stable=True).indices[:, :k]
    q = p.gather(1, ids)
    return ids, q / q.sum(1, keepdim=True)


@pytest.mark.parametrize("E", [32, 64, 96, 100, 128, 160, 320, 384, 512])
def test_gate_finite_logits_far_below_zero_set_no_flag(E):
    logits, sb = _far_logits(E), (torch.arange(E) % 7).float() * -0.125
    sb[5:9] = 0.5  # (distinct from the next by far more than a softmax of equal logits)
    ids, w = _softmax_choice(logits, sb, 4)
    got, gw = _gate(logits.cuda(), sb.cuda(), 4, moe.make_gate("softmax"), flags=0)
    for t in (0, 1, 2, 5):  # (equal scores in the others: order and weights hang on the last bits of a softmax)
        assert got[t].tolist() == ids[t].tolist() == [5, 6, 7, 8]
        _within(gw[t].cpu(), w[t], w[t] * W_REL)
    assert bool(gw.isfinite().all()) and bool(((gw.sum(1) - 1).abs() < 1e-6).all())


@pytest.mark.parametrize("E", [96, 160, 320, 512])
@pytest.mark.parametrize("fused", [1, 2])
@pytest.mark.parametrize("T", [3, 130])
def test_gate_from_rows_with_logits_far_below_zero_sets_no_flag(E, fused, T):
    x, Wg = torch.zeros((T, 256), dtype=BF16, device="cuda"), torch.zeros((256, E), dtype=BF16, device="cuda")
    sb = torch.zeros(E, device="cuda")
    sb[5:9] = 0.5
    old = moe.moe_set_option(moe.MOE_OPT_FUSED_ROUTING, fused)
    try:
        for far in (-100.0, torch.finfo(F32).min):
            lb = torch.full((E,), far, device="cuda")
            got, gw = _gate(torch.empty((T, E), device="cuda"), sb, 4, moe.make_gate("softmax"), x=x, Wg=Wg, lb=lb, flags=0)
            assert bool((got == torch.tensor([5, 6, 7, 8], device="cuda")).all()) and bool(((gw - 0.25).abs() < 1e-6).all())
    finally:
        moe.moe_set_option(moe.MOE_OPT_FUSED_ROUTING, old)


@pytest.mark.parametrize("mask", [-math.inf, math.inf, math.nan])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("kw", [dict(), dict(score="softmax"), dict(n_group=8, topk_group=2), dict(score="softmax", n_group=8, topk_group=2, group_score="max")],
                         ids=["sigmoid", "softmax", "sigmoid-groups", "softmax-groups"])
def test_gate_experts_masked_by_the_bias_weigh_nothing(kw, renorm, mask):
    """A bias that is not finite takes its expert out: chosen last, weight 0, whatever its logit;
    a token that has only such experts to choose gets equal weights."""
    E, k = 64, 4
    logits = torch.linspace(-2, 2, E).repeat(3, 1)
    logits[1] = logits[1].flip(0)
    logits[2, :30] = -60.0
    for left in (0, 1, 2, 3, 20):
        sb = torch.full((E,), mask)
        sb[7:7 + left] = 0.25
        out = torch.where(sb.isfinite(), logits, torch.full_like(logits, -math.inf))
        ids, w, _ = ref.gate(out, torch.where(sb.isfinite(), sb, torch.zeros(E)), k, renorm=renorm, scale=2.0, **kw)
        if not renorm and left and kw.get("score") == "softmax":  # the softmax is over all finite logits
            w = 2.0 * torch.softmax(logits.double(), dim=1).gather(1, ids) * sb.isfinite()[ids]
        got, gw = _gate(logits.cuda(), sb.cuda(), k, moe.make_gate(scale=2.0, **kw), renorm, flags=moe.MOE_DEV_NONFINITE_LOGIT)
        assert got.tolist() == ids.tolist(), left
        _within(gw.cpu(), w, w * W_REL)
        assert bool((gw.cpu()[~sb.isfinite()[ids]] == (0 if left else 2.0 / k)).all())


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", False)])
def test_gate_weights_are_quotients(score, renorm):
    """Weights as expf and division have them: half an ulp (and 2^-20 of one) from the quotient
    of fp32 numbers, which torch's exp, the same function, gives here, its sum added in pairs 4,
    2 and 1 lanes apart as the kernel adds it."""
    T, E, k = 20000, 128, 8
    logits = _normal((T, E), 3, _gen(11), F32)
    ids, w = _gate(logits, None, k, moe.make_gate(score), renorm)
    x = logits.gather(1, ids.long())
    if score == "sigmoid":
        p, z = torch.ones_like(x), 1 + torch.exp(-x)
    else:
        z = p = torch.exp(x - x[:, :1])
        for o in (4, 2, 1):
            z = z[:, :o] + z[:, o:2 * o]
    want = p.double() / z.double()
    ulp = 2.0 ** (torch.floor(torch.log2(want)) - 23)
    _within(w, want, ulp * 0.5 * (1 + 2.0 ** -19))


# ------------------------------------------------------------------- lora
@pytest.mark.parametrize("T", [1, 5, 32, 40, 100, 1024])
@pytest.mark.parametrize("r", [8, 16, 24, 40])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_lora_infinite_rows_stay_infinite(T, r, dt):
    """An infinity of x times positive A and B is one in y (ranks that a kernel pads bring no
    0 times infinity), and leaves the other rows alone."""
    K = N = 64
    g = _gen(T + r)
    x = _normal((T, K), 1, g).abs()
    A, B = _normal((1, r, K), 0.1, g).abs() + 0.01, _normal((1, N, r), 0.1, g).abs() + 0.01
    ids, base = torch.zeros(T, dtype=torch.int32, device="cuda"), _normal((T, N), 1, g, dt)
    ws = torch.zeros(moe.moe_lora_workspace_size(T, K, N, r, 1), dtype=torch.uint8, device="cuda")
    before, y = torch.empty_like(base), torch.empty_like(base)
    moe.moe_lora(T, K, N, r, 1, x, ids, A, B, None, base, before, ws)
    x[T // 2, 9] = math.inf
    moe.moe_lora(T, K, N, r, 1, x, ids, A, B, None, base, y, ws)
    assert bool((y[T // 2] == math.inf).all())
    before[T // 2] = math.inf
    assert torch.equal(y, before)


def test_lora_in_the_workspace_of_a_larger_batch():
    """One workspace, of the size for the most rows, takes every smaller batch."""
    for K, N, r, n, most in ((1032, 264, 64, 1, 2100), (520, 264, 40, 20, 1400), (264, 136, 128, 70, 2600)):
        g = _gen(K + n)
        x, A, B = _normal((most, K), 1, g), _normal((n, r, K), 0.1, g), _normal((n, N, r), 0.1, g)
        ids, base = torch.randint(-1, n, (most,), device="cuda", generator=g).int(), _normal((most, N), 1, g)
        size = moe.moe_lora_workspace_size(most, K, N, r, n)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        for T in (most, 1023, 1024, 700, 300, 65, 64, 33, 1, most):
            y = torch.empty((T, N), dtype=BF16, device="cuda")
            moe.moe_lora(T, K, N, r, n, x, ids, A, B, None, base, y, ws)
            y64, allowed = ref.lora(x[:T], ids[:T], A, B, None, base[:T], BF16)
            _within(y, y64, allowed)
        assert moe.moe_read_device_status(ws) == 0


# ------------------------------------------------------------------ block
@pytest.mark.parametrize("w", ["bf16", "nk", "a8"])
def test_block_in_the_workspace_of_a_larger_batch(w):
    """Batches that run moe_layer's kernels, in a workspace without the few-token scratch, as in
    one of their own: the same bits, and nothing written behind it."""
    D, E, k, I, Is = 512, 64, 4, 128, 128
    gate = moe.make_gate(n_group=8, topk_group=4, scale=2.5)
    n = moe.moe_workspace_size(moe.make_config(64, D, E, k, I, Is, **WD[w]))
    ws = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    ws[n:] = 173
    for T in (64, 17, 24, 32, 40):
        d = _block_inputs(w, T, D, E, k, I, Is, seed=T)
        cfg = moe.make_config(T, D, E, k, I, Is, **WD[w])
        want = _block(cfg, gate, d, moe.alloc_workspace(cfg))
        assert all(torch.equal(a, b) for a, b in zip(_block(cfg, gate, d, ws[:n]), want))
    assert moe.moe_read_device_status(ws[:n]) == 0 and bool((ws[n:] == 173).all())
