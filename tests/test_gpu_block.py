"""moe_add_rms_norm, moe_route_gated, moe_lora and moe_block on the GPU, against
plain 64-bit implementations with derived error bounds (_block_ref)."""
import math

import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests import _block_ref as ref
from tests import _few_ref as few
from tests._lib import ensure_library

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, std, g, dtype=BF16):
    return torch.empty(shape, device="cuda").normal_(0, std, generator=g).to(dtype)


def _within(got, want, allowed):
    got = got.double()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= allowed)  # (NaN is bad)
    assert not bool(bad.any()), f"{int(bad.sum())} values off, the first by {float((got - want).abs()[bad][0]):.3e} " \
                                f"of {float(allowed[bad][0]):.3e} allowed, at {bad.nonzero()[0].tolist()}"


# ------------------------------------------------------------------- norm
def _check_norm(x, res, w, eps, want_sum=True, want_y=True, group=-1, in_place=None):
    T, D = x.shape
    s64, y64, rel = ref.norm(x, res, w, eps)
    kept = x.clone(), None if res is None else res.clone()
    nan = lambda dt: torch.full((T, D), float("nan"), dtype=dt, device="cuda")  # noqa: E731
    sum_out, y = nan(x.dtype) if want_sum else None, nan(x.dtype) if want_y else None
    if in_place:
        sum_out, y = (x, res) if in_place == "sum" else (res, x)
    q = scales = None
    if group >= 0:
        q = torch.zeros((T, D), dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.full((T, D // (group or D)), float("nan"), device="cuda")
    moe.moe_add_rms_norm(T, D, x, res, w, eps, sum_out, y, q, scales, max(group, 0))
    if sum_out is not None:
        _within(sum_out, s64, ref.rounded(s64, x.dtype, ref.U))
    if y is not None:
        _within(y, y64, ref.rounded(y64, x.dtype, rel))
    if group >= 0:
        s, wide, allowed = ref.e4m3(y64, group, rel)
        _within(scales, s, s * (rel + 2 * ref.U))
        _within(q.double() * scales.double().repeat_interleave(group or D, dim=1), y64, allowed)
    if not in_place:
        assert torch.equal(x, kept[0]) and (res is None or torch.equal(res, kept[1]))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(1, 8), (1, 2048), (3, 264), (5, 1024), (2, 1032), (77, 2816), (9, 8192), (3, 16384), (2, 32768),
                                 (4000, 256), (700, 4104), (400, 16392)])
def test_norm(T, D, dtype):
    g = _gen(T * 7 + D)
    x, res = _normal((T, D), 1, g, dtype), _normal((T, D), 3, g, dtype)
    w = (1 + _normal((D,), 0.3, g, F32)).to(dtype)
    _check_norm(x, res, w, 1e-6, group=0)
    _check_norm(x, None, w, 1e-5, want_sum=False)
    _check_norm(x, res, w, 0.0, want_y=False, group=0)
    for in_place in ("sum", "y"):
        _check_norm(x.clone(), res.clone(), w, 1e-6, in_place=in_place)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,D", [(1, 128), (3, 384), (33, 2816), (5, 1152), (2, 32768), (300, 7168)])
def test_norm_group_scales(T, D, group):
    g = _gen(T + D + group)
    x = _normal((T, D), 1, g)
    x[:, :group] *= 100  # a group far from the others
    x[0, group - 8:group] = 0
    if D > group:
        x[-1, -group:] = 0  # a group of zeros
    for dtype in (BF16, F32):
        _check_norm(x.to(dtype), None, torch.ones(D, dtype=dtype, device="cuda"), 1e-6, want_sum=False, group=group)


@pytest.mark.parametrize("D", [256, 4096])
def test_norm_rows_at_the_ends_of_the_range(D):
    """Zero rows; squares above and below fp32's range, with and without eps."""
    g = _gen(D)
    rows = [torch.zeros(D, device="cuda")]
    for e in (1e30, 3e37, 1e19, 1e-20, 1e-25, 1e-36):
        rows.append(_normal((D,), 1, g, F32) * e)
    one = torch.zeros(D, device="cuda")
    one[D // 2] = 2e38
    x = torch.stack(rows + [one])
    w = torch.ones(D, device="cuda")
    for eps in (1e-6, 1e-30, 0.0):
        for dtype in (F32, BF16):
            xs = x.to(dtype)
            if eps == 0.0:
                xs = xs[1:]  # 0 / 0
            s64, y64, rel = ref.norm(xs, None, w, eps)
            y = torch.empty_like(xs)
            q, s = torch.empty(xs.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(len(xs), device="cuda")
            moe.moe_add_rms_norm(len(xs), D, xs, None, w.to(dtype), eps, None, y, q, s)
            _within(y, y64, ref.rounded(y64, dtype, rel))
            s64, wide, allowed = ref.e4m3(y64, 0, rel)
            _within(s[:, None], s64, s64 * (rel + 2 * ref.U))
            _within(q.double() * s.double()[:, None], y64, allowed)


def test_norm_infinities_and_nan_stay_in_their_rows():
    g = _gen(5)
    x = _normal((6, 512), 1, g)
    x[1, 7], x[3, 500], x[4, 0] = math.inf, math.nan, -math.inf
    w = torch.ones(512, dtype=BF16, device="cuda")
    y, q, s = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(6, 8, device="cuda")
    moe.moe_add_rms_norm(6, 512, x, None, w, 1e-6, None, y, q, s, 64)
    _, y64, rel = ref.norm(x, None, w, 1e-6)
    good = torch.tensor([0, 2, 5], device="cuda")
    _within(y[good], y64[good], ref.rounded(y64[good], BF16, rel))
    assert bool(y[3].isnan().all()) and bool(y[1, 7].isnan()) and bool(y[4, 0].isnan())
    assert bool((y[1, 8:] == 0).all()) and bool((y[4, 1:] == 0).all())  # finite / infinite
    assert bool(s[3].isnan().all()) and bool(s[1, 0].isnan()) and bool((s[1, 1:] == 1).all())
    assert bool(q[3].float().isnan().all()) and bool(s[good].isfinite().all())


def test_norm_offsets_that_pass_32_bits():
    T, D = 140_000, 16384
    x = torch.empty((T, D), dtype=BF16, device="cuda").normal_(generator=_gen(1))
    w = torch.ones(D, dtype=BF16, device="cuda")
    q, s = torch.empty((T, D), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((T, D // 128), device="cuda")
    y = torch.empty_like(x)
    moe.moe_add_rms_norm(T, D, x, None, w, 1e-6, None, y, q, s, 128)
    for t in (0, T // 2, 131_071, 131_072, T - 1):
        _, y64, rel = ref.norm(x[t:t + 1], None, w, 1e-6)
        _within(y[t:t + 1], y64, ref.rounded(y64, BF16, rel))
        s64, wide, allowed = ref.e4m3(y64, 128, rel)
        _within(q[t:t + 1].double() * s[t:t + 1].double().repeat_interleave(128, dim=1), y64, allowed)


# ------------------------------------------------------------------- gate
def _gate(logits, sb, k, gate, renorm=True, x=None, Wg=None, lb=None, flags=0):
    T, E = logits.shape
    cfg = moe.make_config(T, 8 if x is None else x.shape[1], E, k, 8, renormalize=renorm)
    ws = moe.alloc_workspace(cfg)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    moe.moe_route_gated(cfg, gate, x, Wg, lb, sb, logits, ids, w, ws)
    assert moe.moe_read_device_status(ws) == flags
    return ids, w


GATES = [dict(), dict(score="softmax"), dict(score="softmax", scale=2.5), dict(n_group=8, topk_group=4, scale=2.5),
         dict(n_group=8, topk_group=3, group_score="max"), dict(score="softmax", n_group=4, topk_group=2),
         dict(score="softmax", n_group=16, topk_group=9, group_score="max"), dict(n_group=32, topk_group=31)]


# the allowed relative error of a weight: expf's two ulps and the difference that it is
# taken of (below 8: 8 U), once more in the sum, the sum itself (32 lanes: 6 U), the
# divisions and the factor
W_REL = 40 * ref.U


@pytest.mark.parametrize("gate", range(len(GATES)))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,k", [(32, 1), (64, 4), (128, 8), (160, 6), (256, 8), (320, 9), (384, 16), (512, 10), (512, 16)])
def test_gate_with_ties(E, k, bias, gate):
    """Logits (and biases) of few values, so that many are the same, in every layout of
    groups over a warp's lanes; what differs does so by far more than fp32's error."""
    kw = GATES[gate]
    if kw.get("topk_group", 1) * (E // kw.get("n_group", 1)) < k:
        pytest.skip("fewer experts than k")
    cpu = torch.Generator().manual_seed(E * 31 + k + gate)
    T = 37
    logits = (torch.randint(-64, 65, (T, E), generator=cpu).float() / 16)
    logits[0] = 1.0  # all the same
    logits[1] = -60.0
    sb = (torch.randint(0, 4, (E,), generator=cpu).float() / 4) * (1.0 if kw.get("score", "sigmoid") == "sigmoid" else 1 / E) if bias else None
    for renorm in (True, False):
        ids, w, _ = ref.gate(logits, sb, k, renorm=renorm, **kw)
        got, gw = _gate(logits.cuda(), None if sb is None else sb.cuda(), k, moe.make_gate(**kw), renorm)
        keep = torch.tensor([ref.gate(logits[t:t + 1], sb, k, renorm=renorm, **kw)[2] > 1e-6 * (1.0 if kw.get("score", "sigmoid") == "sigmoid" else 1 / E)
                             for t in range(T)])
        assert int(keep.sum()) >= T - 4  # (sums of a score and a bias can fall together)
        assert torch.equal(got.cpu().long()[keep], ids[keep])
        _within(gw.cpu()[keep], w[keep], w[keep] * W_REL + 1e-38)


@pytest.mark.parametrize("E,k,kw", [(1, 1, {}), (6, 2, dict(n_group=2, topk_group=1)), (7, 7, dict(score="softmax")),
                                    (30, 3, dict(n_group=10, topk_group=4)), (31, 5, dict(n_group=31, topk_group=7)),
                                    (300, 7, dict(score="softmax", n_group=3, topk_group=2))])
def test_gate_odd_sizes(E, k, kw):
    logits = torch.linspace(-3, 3, E).repeat(5, 1)
    logits = torch.stack([row[torch.randperm(E, generator=torch.Generator().manual_seed(i))] for i, row in enumerate(logits)])
    ids, w, margin = ref.gate(logits, None, k, **kw)
    assert margin > 1e-6
    got, gw = _gate(logits.cuda(), None, k, moe.make_gate(**kw))
    assert torch.equal(got.cpu().long(), ids)
    _within(gw.cpu(), w, w * W_REL)


def test_gate_non_finite_logits():
    """They are chosen last, groups of them too; a token with nothing else gets equal weights."""
    E, k = 64, 4
    logits = torch.linspace(-2, 2, E).repeat(6, 1)
    logits[0, 40:] = math.nan
    logits[1, :] = -math.inf
    logits[2, 60], logits[2, 3] = math.inf, -math.inf
    logits[3, 2:] = math.nan  # fewer finite ones than k
    logits[4, 8:] = torch.finfo(F32).min  # a mask's lowest value is a number
    for kw in (dict(), dict(score="softmax"), dict(n_group=8, topk_group=2), dict(score="softmax", n_group=8, topk_group=2, group_score="max")):
        for sb in (None, torch.full((E,), 0.25)):
            ids, w, _ = ref.gate(logits, sb, k, scale=2.0, **kw)
            got, gw = _gate(logits.cuda(), None if sb is None else sb.cuda(), k, moe.make_gate(scale=2.0, **kw), flags=moe.MOE_DEV_NONFINITE_LOGIT)
            assert torch.equal(got.cpu().long(), ids), kw
            _within(gw.cpu(), w, w * W_REL)
    sb = torch.zeros(E)
    sb[5] = math.nan
    got, _ = _gate(logits[5:].cuda(), sb.cuda(), k, moe.make_gate(), flags=moe.MOE_DEV_NONFINITE_LOGIT)
    assert got.tolist() == [[63, 62, 61, 60]]


def test_gate_small_sigmoids_keep_their_ratios():
    logits = torch.tensor([[-100.0, -101.5, -99.0, -140.0] + [-200.0] * 28, [-59.0, -60.5, -63.0, -58.0] + [-80.0] * 28])
    ids, w, _ = ref.gate(logits, None, 3)
    got, gw = _gate(logits.cuda(), None, 3, moe.make_gate())
    assert torch.equal(got.cpu().long(), ids)
    _within(gw.cpu(), w, w * W_REL)


@pytest.mark.parametrize("T,D,E,k", [(1, 256, 64, 4), (40, 2048, 128, 8), (65, 512, 256, 8), (300, 1024, 512, 10), (4100, 512, 128, 8),
                                     (2100, 768, 320, 6)])
@pytest.mark.parametrize("fused", [1, 2])
def test_gate_from_rows(T, D, E, k, fused):
    """Through the projection: the logits within their error, ids and weights as the
    kernel's own logits have them."""
    g = _gen(T + E)
    x, Wg = _normal((T, D), 1, g), _normal((D, E), 0.05, g)
    lb, sb = _normal((E,), 1, g, F32), _normal((E,), 0.1, g, F32)
    old = moe.moe_set_option(moe.MOE_OPT_FUSED_ROUTING, fused)
    try:
        for kw in (dict(n_group=8, topk_group=4, scale=2.5), dict(score="softmax")):
            for b, s in ((None, sb), (lb, None)):
                logits = torch.full((T, E), float("nan"), device="cuda")
                ids, w = _gate(logits, s, k, moe.make_gate(**kw), x=x, Wg=Wg, lb=b)
                exact = x.double() @ Wg.double() + (0 if b is None else b.double())
                mag = x.double().abs() @ Wg.double().abs() + (0 if b is None else b.double().abs())
                _within(logits, exact, (D + 20) * 2 * ref.U * mag)
                again, w2 = _gate(logits.clone(), s, k, moe.make_gate(**kw))
                assert torch.equal(ids, again) and torch.equal(w, w2)
                rows = list(range(min(T, 40)))
                for t in rows:
                    want, ww, margin = ref.gate(logits[t:t + 1].cpu(), None if s is None else s.cpu(), k, **kw)
                    if margin > 1e-6 / (1 if kw.get("score", "sigmoid") == "sigmoid" else E):
                        assert ids[t].tolist() == want[0].tolist()
                        _within(w[t:t + 1].cpu(), ww, ww * W_REL)
    finally:
        moe.moe_set_option(moe.MOE_OPT_FUSED_ROUTING, old)


@pytest.mark.parametrize("T,D,E,k", [(5, 64, 30, 3), (70, 72, 7, 7), (33, 256, 512, 16)])
def test_gate_from_rows_in_32_bits(T, D, E, k):
    g = _gen(E)
    x, Wg, sb = _normal((T, D), 1, g, F32), _normal((D, E), 0.1, g, F32), _normal((E,), 0.2, g, F32)
    cfg = moe.make_config(T, D, E, k, 8, act_dtype="f32", w_dtype="f32")
    ws, logits = moe.alloc_workspace(cfg), torch.empty((T, E), device="cuda")
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    moe.moe_route_gated(cfg, moe.make_gate(), x, Wg, None, sb, logits, ids, w, ws)
    _within(logits, x.double() @ Wg.double(), (D + 20) * 2 * ref.U * (x.double().abs() @ Wg.double().abs()))
    again, w2 = _gate(logits.clone(), sb, k, moe.make_gate())
    assert torch.equal(ids, again) and torch.equal(w, w2)


def test_gate_of_softmax_is_moe_route():
    """Without bias, groups and factor the choice is moe_route's."""
    for T, E, k in ((3, 48, 5), (100, 128, 8), (257, 512, 10)):
        logits = _normal((T, E), 2, _gen(E), F32)
        for renorm in (True, False):
            cfg = moe.make_config(T, 8, E, k, 8, renormalize=renorm)
            ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
            moe.moe_route(cfg, None, None, None, logits, ids, w, moe.alloc_workspace(cfg))
            got, gw = _gate(logits, None, k, moe.make_gate("softmax"), renorm)
            assert torch.equal(ids, got)
            _within(gw, w.double(), w.double() * 2 * W_REL)


# ------------------------------------------------------------------- lora
def _lora_inputs(T, K, N, r, n, dt, seed, how):
    g = _gen(seed)
    d = dict(x=_normal((T, K), 1, g), A=_normal((n, r, K), 0.05, g), B=_normal((n, N, r), 0.1, g),
             scales=torch.empty(n, device="cuda").uniform_(0.5, 2, generator=g), base=_normal((T, N), 1, g, dt))
    ids = torch.randint(-1, n, (T,), device="cuda", generator=g)
    if how == "runs":
        ids = ids.sort().values
    if how == "one":
        ids = torch.full_like(ids, n - 1)
    if how == "none":
        ids = torch.full_like(ids, -1)
    d["ids"] = ids.int()
    return d


def _lora(d, y, base, scales=True):
    T, K = d["x"].shape
    n, N, r = d["B"].shape
    ws = torch.full((moe.moe_lora_workspace_size(T, K, N, r, n),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_lora(T, K, N, r, n, d["x"], d["ids"], d["A"], d["B"], d["scales"] if scales else None, base, y, ws)
    return y


def _check_lora(d, dt, base=True, scales=True, in_place=False):
    T, N = d["x"].shape[0], d["B"].shape[1]
    b = d["base"] if base else None
    y64, allowed = ref.lora(d["x"], d["ids"], d["A"], d["B"], d["scales"] if scales else None, b, dt)
    y = b.clone() if in_place else torch.full((T, N), float("nan"), dtype=dt, device="cuda")
    _lora(d, y, y if in_place else b, scales)
    _within(y, y64, allowed)
    # the bound above adds up the magnitudes of long sums.  An mma step of 16 terms truncates
    # its sum by less than an ulp, half of one on average (2^-24): K / 128 steps to a warp at
    # most, then its 8 warps' sums and the planes, 3 r / 16 steps of the second product
    (n, r, K), off, size = d["A"].shape, float((y.double() - y64).norm()), float(y64.norm())
    assert off <= size * (2.0 ** -8 if dt == BF16 else (K / 128 + 3 * r / 16 + 16) * ref.U) + 1e-30
    bare = ~((d["ids"] >= 0) & (d["ids"] < d["A"].shape[0]))
    assert torch.equal(y[bare], b[bare] if base else torch.zeros_like(y[bare]))
    return y


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T,K,N,r,n,how", [
    (1, 8, 8, 8, 1, "one"), (1, 2048, 2048, 16, 8, "one"), (1, 2056, 520, 16, 3, "mixed"), (5, 1000, 520, 32, 4, "mixed"),
    (32, 1024, 264, 24, 2, "mixed"), (31, 4096, 1032, 8, 31, "mixed"), (33, 256, 264, 16, 4, "mixed"), (30, 512, 40, 16, 3, "none"), (2, 264, 40, 24, 2, "mixed"), (17, 1000, 1032, 8, 1, "one"),
    (33, 512, 264, 64, 3, "mixed"), (61, 1024, 520, 64, 40, "mixed"), (64, 256, 512, 128, 64, "mixed"), (64, 256, 256, 72, 2, "none"),
    (65, 256, 264, 16, 1, "one"), (100, 328, 776, 40, 90, "mixed"), (129, 512, 256, 32, 2, "runs"), (300, 256, 1544, 256, 5, "mixed"),
    (1000, 512, 320, 64, 4, "runs"), (1025, 136, 128, 24, 1, "none"), (2000, 256, 264, 16, 1500, "mixed"), (513, 64, 64, 200, 16, "mixed"),
    (700, 520, 1288, 96, 6, "mixed"), (400, 264, 136, 128, 2, "runs"), (5000, 1000, 1000, 40, 3, "mixed"), (260, 136, 2056, 16, 2, "mixed"),
    (3000, 4104, 72, 8, 7, "runs"), (90, 72, 8, 256, 1, "one"), (1024, 64, 64, 200, 16, "mixed"), (1500, 256, 1544, 256, 5, "mixed"),
    (1100, 520, 1288, 96, 6, "mixed"), (2100, 264, 136, 128, 2, "runs"), (1300, 136, 2056, 16, 2, "mixed"), (1024, 72, 8, 256, 1, "one"),
    (9000, 200, 104, 16, 30, "mixed"), (1024, 2048, 64, 256, 2, "mixed"), (1030, 4104, 72, 136, 1, "one"), (1100, 1032, 200, 64, 9, "mixed"),
    (64, 1000, 520, 24, 1, "one"), (49, 264, 264, 128, 2, "runs"), (64, 2048, 520, 64, 3, "mixed"), (32, 1024, 264, 16, 1, "one"),
    (2049, 512, 264, 32, 64, "mixed"), (1023, 512, 264, 32, 2, "mixed")])
def test_lora(T, K, N, r, n, how, dt):
    d = _lora_inputs(T, K, N, r, n, dt, T + K + N + r, how)
    y = _check_lora(d, dt)
    assert torch.equal(y, _check_lora(d, dt))  # the same bits
    assert torch.equal(y, _check_lora(d, dt, in_place=True))
    _check_lora(d, dt, base=False, scales=False)


def test_lora_ids_out_of_range_are_rows_without_an_adapter():
    for T in (50, 400, 1400):
        d = _lora_inputs(T, 128, 64, 16, 3, F32, T, "mixed")
        d["ids"][::5] = 3
        d["ids"][1::7] = -(2 ** 31)
        d["ids"][2::9] = 2 ** 31 - 1
        _check_lora(d, F32)
        _check_lora(d, F32, in_place=True)


def test_lora_rows_do_not_depend_on_their_neighbours():
    """A row gets the same bits wherever it stands among others of the batch's size; an
    infinity stays in its row."""
    for T in (60, 500, 1100):
        d = _lora_inputs(T, 520, 264, 24, 6, BF16, T, "mixed")
        y = _lora(d, torch.empty_like(d["base"]), d["base"])
        p = torch.randperm(T, device="cuda", generator=_gen(3))
        e = dict(d, x=d["x"][p].contiguous(), ids=d["ids"][p].contiguous(), base=d["base"][p].contiguous())
        assert torch.equal(_lora(e, torch.empty_like(y), e["base"]), y[p])
        d["x"][7, 100], d["x"][9, 3] = math.inf, math.nan
        z = _lora(d, torch.empty_like(y), d["base"])
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[7] = rest[9] = False
        assert torch.equal(z[rest], y[rest])


def test_lora_large_products_stay_infinite():
    """x A^T past bf16's range: no NaN from its terms."""
    for T in (4, 1024):
        d = _lora_inputs(T, 64, 64, 8, 1, F32, 1, "one")
        d["x"].fill_(1e30)
        d["A"].fill_(1e30)
        d["B"].fill_(1.0)
        assert bool((_lora(d, torch.empty_like(d["base"]), d["base"]) == math.inf).all())


def test_lora_calls_in_a_row_see_what_the_last_wrote():
    """Calls of many sizes in one workspace, with B, ids and the base changed between them by
    kernels of the same stream and nothing waited for: the bits of the same calls made one by
    one without programmatic launches."""
    g = _gen(8)
    K, N, r, n = 264, 1032, 40, 9
    A, B0 = _normal((n, r, K), 0.05, g), _normal((n, N, r), 0.1, g)
    sizes = [3, 2000, 64, 65, 1, 1024, 300, 5000, 1500, 17] * 3
    x, base0 = _normal((5000, K), 1, g), _normal((5000, N), 1, g)
    every = [torch.randint(-1, n, (T,), device="cuda", generator=g).int() for T in sizes]
    ws = torch.zeros(max(moe.moe_lora_workspace_size(T, K, N, r, n) for T in sizes), dtype=torch.uint8, device="cuda")

    def run(wait):
        B, ids, base, got = B0.clone(), torch.empty(5000, dtype=torch.int32, device="cuda"), base0.clone(), []
        for T, i in zip(sizes, every):
            B.neg_()
            ids[:T].copy_(i)
            base.mul_(0.5)
            y = torch.empty((T, N), dtype=BF16, device="cuda")
            moe.moe_lora(T, K, N, r, n, x, ids, A, B, None, base, y, ws)
            moe.moe_lora(T, K, N, r, n, x, ids, A, B, None, base, base, ws)
            got.append(y)
            if wait:
                torch.cuda.synchronize()
        return got + [base]

    got = run(False)
    old = moe.moe_set_option(moe.MOE_OPT_PDL, 0)
    try:
        want = run(True)
    finally:
        moe.moe_set_option(moe.MOE_OPT_PDL, old)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_lora_offsets_that_pass_32_bits():
    """A and B past 2^32 bytes, x and y past 2^31 values."""
    g = _gen(2)
    n, r, K, N, T = 600, 64, 65536, 32768, 40_000
    d = dict(x=torch.empty((T, K), dtype=BF16, device="cuda").normal_(generator=g),
             A=torch.empty((n, r, K), dtype=BF16, device="cuda").normal_(0, 0.01, generator=g),
             B=torch.empty((n, N, r), dtype=BF16, device="cuda").normal_(0, 0.1, generator=g),
             scales=torch.ones(n, device="cuda"), base=torch.zeros((T, N), dtype=BF16, device="cuda"))
    d["ids"] = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 5, 20_000, 32_767, 32_768, 39_999], device="cuda")
    d["ids"][rows] = torch.tensor([0, 511, 599, 512, 300, 599], dtype=torch.int32, device="cuda")
    y = _lora(d, torch.empty_like(d["base"]), d["base"])
    y64, allowed = ref.lora(d["x"][rows], d["ids"][rows], d["A"], d["B"], d["scales"], d["base"][rows], BF16)
    _within(y[rows], y64, allowed)
    few = dict(d, x=d["x"][rows].contiguous(), ids=d["ids"][rows].contiguous(), base=d["base"][rows].contiguous())
    _within(_lora(few, torch.empty_like(few["base"]), few["base"]), y64, allowed)  # the few-row kernels
    d["ids"][rows] = -1
    bare = d["ids"] == -1
    y[rows] = 0
    assert not bool(y[bare].any())


def test_no_workspace_is_refused():
    """None for ws: the library's error, as the other calls have it, and nothing written."""
    g = _gen(3)
    T, K, N, r, n = 3, 64, 24, 8, 2
    x, A, B = _normal((T, K), 1, g), _normal((n, r, K), 1, g), _normal((n, N, r), 1, g)
    ids, y = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.full((T, N), 7.0, dtype=BF16, device="cuda")
    cfg = moe.make_config(T, K, 16, 2, 16)
    logits, chosen, w = _normal((T, 16), 1, g, F32), torch.full((T, 2), -3, dtype=torch.int32, device="cuda"), torch.empty((T, 2), device="cuda")
    with pytest.raises(moe.MoEError, match="workspace"):
        moe.moe_lora(T, K, N, r, n, x, ids, A, B, None, None, y, None)
    with pytest.raises(moe.MoEError, match="workspace"):
        moe.moe_route_gated(cfg, moe.make_gate(), None, None, None, None, logits, chosen, w, None)
    W13, W2, Wg = _normal((16, K, 32), 1, g), _normal((16, 16, K), 1, g), _normal((K, 16), 1, g)
    out = torch.full_like(x, 7.0)
    with pytest.raises(moe.MoEError, match="workspace"):
        moe.moe_block(cfg, None, x, None, None, 0.0, Wg, None, None, W13, None, W2, None, None, None, None, None, None, None, out, None)
    assert bool((y == 7).all()) and bool((out == 7).all()) and bool((chosen == -3).all())


# ------------------------------------------------------------------ block
def _weights(w, lead, K, N, g):
    W = torch.empty((*lead, K, N), device="cuda").normal_(0, 0.05, generator=g)
    if w in ("bf16", "f32"):
        return W.to(BF16 if w == "bf16" else F32), None
    s = W.abs().amax(-2) / 448
    q = (W / s.unsqueeze(-2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (q if w == "fp8_e4m3" else q.transpose(-1, -2).contiguous()), s


def _block_inputs(w, T, D, E, k, I, Is, seed=0):
    g = _gen(seed)
    dt = F32 if w == "f32" else BF16
    d = dict(x=_normal((T, D), 1, g, dt), residual=_normal((T, D), 2, g, dt), nw=(1 + _normal((D,), 0.2, g, F32)).to(dt),
             Wg=_normal((D, E), 0.05, g, dt), sb=_normal((E,), 0.1, g, F32), lb=_normal((E,), 0.5, g, F32))
    d["W13"], d["s13"] = _weights(w, (E,), D, 2 * I, g)
    d["W2"], d["s2"] = _weights(w, (E,), I, D, g)
    d["W13s"], d["s13s"] = _weights(w, (), D, 2 * Is, g) if Is else (None, None)
    d["W2s"], d["s2s"] = _weights(w, (), Is, D, g) if Is else (None, None)
    return d


def _block(cfg, gate, d, ws, norm=True, sb=True, stream=None):
    T, D = d["x"].shape
    dt = d["x"].dtype
    sum_out, y = (torch.empty_like(d["x"]), torch.empty_like(d["x"])) if norm else (None, None)
    out = torch.full((T, D), float("nan"), dtype=dt, device="cuda")
    moe.moe_block(cfg, gate, d["x"], d["residual"] if norm else None, d["nw"] if norm else None, 1e-6 if norm else 0.0, d["Wg"], d["lb"],
                  d["sb"] if sb else None, d["W13"], d["s13"], d["W2"], d["s2"], d["W13s"], d["s13s"], d["W2s"], d["s2s"], sum_out, y,
                  out, ws, stream)
    return sum_out, y, out


WD = {"f32": dict(act_dtype="f32", w_dtype="f32"), "bf16": dict(w_dtype="bf16"), "fp8_e4m3": dict(w_dtype="fp8_e4m3"),
      "nk": dict(w_dtype="fp8_e4m3_nk"), "a8": dict(w_dtype="fp8_e4m3_nk_a8")}


@pytest.mark.parametrize("w", ["f32", "bf16", "fp8_e4m3", "nk", "a8"])
@pytest.mark.parametrize("T,D,E,k,I,Is", [(1, 256, 64, 4, 128, 128), (50, 512, 64, 6, 256, 0), (2100, 512, 128, 8, 128, 256)])
def test_block_is_its_stages(w, T, D, E, k, I, Is):
    """moe_block's sum, normed rows, choice and output are those of moe_add_rms_norm,
    moe_route_gated and the stage calls on them: bit for bit up to the experts, whose GEMMs
    may take other tiles."""
    d = _block_inputs(w, T, D, E, k, I, Is)
    gate = moe.make_gate(n_group=8, topk_group=4, scale=2.5)
    cfg = moe.make_config(T, D, E, k, I, Is, **WD[w])
    ws = moe.alloc_workspace(cfg)
    sum_out, y, out = _block(cfg, gate, d, ws)
    assert moe.moe_read_device_status(ws) == 0
    ids = moe.workspace_view(ws, cfg, "topk_ids", (T, k), torch.int32).clone()
    wt = moe.workspace_view(ws, cfg, "topk_w", (T, k), F32).clone()
    s2, y2 = torch.empty_like(sum_out), torch.empty_like(y)
    q, qs = torch.empty((T, D), dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_add_rms_norm(T, D, d["x"], d["residual"], d["nw"], 1e-6, s2, y2, q, qs)
    assert torch.equal(sum_out, s2) and torch.equal(y, y2)
    if w == "a8":
        assert torch.equal(moe.workspace_view(ws, cfg, "x16", (T, D), torch.uint8), q)
        assert torch.equal(moe.workspace_view(ws, cfg, "tok_inv", (T,), F32), qs)
    ws2 = moe.alloc_workspace(cfg)
    logits = torch.empty((T, E), device="cuda")
    ids2, wt2 = torch.empty_like(ids), torch.empty_like(wt)
    moe.moe_route_gated(cfg, gate, y, d["Wg"], d["lb"], d["sb"], logits, ids2, wt2, ws2)
    assert torch.equal(ids, ids2) and torch.equal(wt, wt2)
    counts, offsets = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rows, dest = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32, device="cuda")
    xp = torch.empty((T * k, D), dtype=y.dtype, device="cuda")
    moe.moe_permute(cfg, ids, y, counts, offsets, rows, dest, xp, ws2)
    hb, yb = (4, 4) if w in ("f32", "bf16") else (4, 2) if w == "fp8_e4m3" else (2, 2)
    buf = lambda n, b: torch.empty(n * b, dtype=torch.uint8, device="cuda")  # noqa: E731
    h, yp = buf(T * k * I, hb), buf(T * k * D, yb)
    hs, so = (buf(T * Is, hb), buf(T * D, yb)) if Is else (None, None)
    moe.moe_grouped_ffn(cfg, xp, offsets, d["W13"], d["s13"], d["W2"], d["s2"], h, yp, y if Is else None, d["W13s"], d["s13s"], d["W2s"],
                        d["s2s"], hs, so, ws2)
    out2 = torch.empty_like(out)
    moe.moe_finalize(cfg, yp, dest, wt, so, out2, ws2)
    if w == "a8":
        # each activation of x is off by half a step of e4m3 on one side, by that and bf16's
        # on the other: 2^-4 + 2^-8 of it at most between the two, 2^-5 as a root of mean
        # squares; h's likewise.  Two products of such factors, of independent signs
        rms = float(out2.double().square().mean().sqrt())
        assert float((out.double() - out2.double()).square().mean().sqrt()) <= 2 ** -4 * rms
    else:
        tol = (2.0 ** -8 if w != "f32" else 2.0 ** -20) * float(out2.double().square().mean().sqrt())
        assert float((out.double() - out2.double()).square().mean().sqrt()) <= tol


@pytest.mark.parametrize("w", ["f32", "bf16", "nk", "a8"])
def test_block_without_norm_and_gate_is_moe_layer(w):
    T, D, E, k, I = 70, 512, 64, 6, 256
    d = _block_inputs(w, T, D, E, k, I, 128)
    cfg = moe.make_config(T, D, E, k, I, 128, **WD[w])
    ws = moe.alloc_workspace(cfg)
    _, _, out = _block(cfg, None, d, ws, norm=False, sb=False)
    want = torch.empty_like(out)
    moe.moe_layer(cfg, d["x"], d["Wg"], d["lb"], d["W13"], d["s13"], d["W2"], d["s2"], d["W13s"], d["s13s"], d["W2s"], d["s2s"], want, ws)
    assert torch.equal(out, want)


def _few_expected(d, kind, y, ids, w, act):
    """(out, allowed error) of a few-token layer for rows y, the chosen experts and their weights."""
    x = y.double().cpu()
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    cpu = {m: None if v is None else v.cpu() for m, v in d.items()}
    k = ids.shape[1]
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        one = lambda s: None if s is None else s[e]  # noqa: E731
        f, ef = few._ffn(x[t], few.dense(cpu["W13"][e], one(cpu["s13"]), kind), few.dense(cpu["W2"][e], one(cpu["s2"]), kind), act,
                         kind != "bf16")
        out.index_put_((t,), w[t, j, None] * f, accumulate=True)
        err.index_put_((t,), w[t, j, None] * (ef + (k + 2) * few.U32 * f.abs()), accumulate=True)
    if cpu["W13s"] is not None:
        f, ef = few._ffn(x, few.dense(cpu["W13s"], cpu["s13s"], kind), few.dense(cpu["W2s"], cpu["s2s"], kind), act, kind != "bf16")
        out, err = out + f, err + ef + 2 * few.U32 * (f.abs() + out.abs())
    return out, err + few.BF16 * (out.abs() + err)


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_nk", "w4_g32", "w4_g64", "w4_g128"])
@pytest.mark.parametrize("T,k,Is", [(1, 4, 128), (8, 6, 0), (13, 3, 256), (32, 4, 128)])
def test_block_of_a_few_tokens(kind, T, k, Is):
    """4-bit weights with the choice by scores, and the other types where moe_layer_few's kernel
    takes them: that kernel's output for the choice that moe_route_gated makes of the normed rows;
    without a gate, moe_layer_few's bits."""
    D, E, I = 512, 64, 256
    if T > {"bf16": 8, "fp8_e4m3_nk": 16}.get(kind, 32):
        pytest.skip("moe_layer's kernels")  # (with a gate bf16 from 5 tokens on: as precise)
    w4 = kind.startswith("w4")
    d = _block_inputs("bf16" if kind == "bf16" or w4 else "fp8_e4m3" if kind == "fp8_e4m3" else "nk", T, D, E, k, I, Is, seed=T)
    if w4:
        for i, (m, s) in enumerate((("W13", "s13"), ("W2", "s2"), ("W13s", "s13s"), ("W2s", "s2s"))):
            if d[m] is not None:
                lead, width = ((E,), I) if i < 2 else ((), Is)
                W, _ = _weights("bf16", lead, *((D, 2 * width) if "13" in m else (width, D)), _gen(T + i))
                d[m], d[s] = moe.quantize_w4(W, int(kind[4:]))
    cfg = moe.make_config(T, D, E, k, I, Is, w_dtype=kind)
    gate = moe.make_gate(n_group=8, topk_group=4, scale=2.5)
    ws = moe.alloc_workspace(cfg)
    sum_out, y, out = _block(cfg, gate, d, ws)
    assert moe.moe_read_device_status(ws) == 0
    ids = moe.workspace_view(ws, cfg, "topk_ids", (T, k), torch.int32).clone()
    w = moe.workspace_view(ws, cfg, "topk_w", (T, k), F32).clone()
    ws2 = moe.alloc_workspace(cfg)
    logits, ids2, w2 = torch.empty((T, E), device="cuda"), torch.empty_like(ids), torch.empty_like(w)
    moe.moe_route_gated(cfg, gate, y, d["Wg"], d["lb"], d["sb"], logits, ids2, w2, ws2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    want, allowed = _few_expected(d, kind, y, ids.long().cpu(), w.double().cpu(), "swiglu")
    _within(out.cpu(), want, allowed)
    assert torch.equal(out, _block(cfg, gate, d, ws)[2])
    _, y, out = _block(cfg, None, d, ws, sb=False)
    want = torch.empty_like(out)
    moe.moe_layer_few(cfg, y, d["Wg"], d["lb"], d["W13"], d["s13"], d["W2"], d["s2"], d["W13s"], d["s13s"], d["W2s"], d["s2s"], want, ws2)
    assert torch.equal(out, want)


def test_block_against_64_bits():
    """The whole block on the oracle's arithmetic: norm, choice and experts in 64 bits."""
    T, D, E, k, I, Is = 24, 256, 32, 4, 128, 64
    d = _block_inputs("f32", T, D, E, k, I, Is)
    gate = dict(n_group=4, topk_group=2, scale=2.5)
    cfg = moe.make_config(T, D, E, k, I, Is, **WD["f32"])
    ws = moe.alloc_workspace(cfg)
    _, y, out = _block(cfg, moe.make_gate(**gate), d, ws)
    _, y64, _ = ref.norm(d["x"], d["residual"], d["nw"], 1e-6)
    logits = y64 @ d["Wg"].double() + d["lb"].double()
    ids, w, _ = ref.gate(logits.cpu(), d["sb"].cpu(), k, **gate)
    keep = torch.tensor([ref.gate(logits[t:t + 1].cpu(), d["sb"].cpu(), k, **gate)[2] > 1e-5 for t in range(T)])
    assert int(keep.sum()) >= T - 2
    assert torch.equal(moe.workspace_view(ws, cfg, "topk_ids", (T, k), torch.int32).cpu().long()[keep], ids[keep])

    def ffn(x, W13, W2):
        gu = x @ W13.double()
        g, u = gu.chunk(2, dim=-1)
        return (g * torch.sigmoid(g) * u) @ W2.double()

    want = ffn(y64, d["W13s"], d["W2s"])
    for t in range(T):
        for j in range(k):
            want[t] += float(w[t, j]) * ffn(y64[t:t + 1], d["W13"][ids[t, j]], d["W2"][ids[t, j]])[0]
    # fp32 throughout: sums of at most 512 terms, 2^-24 each, three deep, of magnitudes a few
    # times the result's
    assert float((out.double() - want)[keep.cuda()].abs().max()) <= 3 * 512 * ref.U * 8 * float(want.square().mean().sqrt())


# ------------------------------------------------------- together, as used
def test_a_served_step():
    """A decode step's pieces in a row, eager, on a stream of its own and replayed from a
    graph: the block, the next norm, a 4-bit projection and its requests' adapters."""
    T, D, E, k, I, N, r, n = 13, 512, 64, 6, 256, 1032, 16, 5
    d = _block_inputs("bf16", T, D, E, k, I, 128)
    gate = moe.make_gate(n_group=8, topk_group=4, scale=2.5)
    cfg = moe.make_config(T, D, E, k, I, 128)
    g = _gen(11)
    qh, sh = moe.quantize_w4(_normal((D, N), 0.05, g), 64)
    ld = _lora_inputs(T, D, N, r, n, F32, 3, "mixed")
    w2 = (1 + _normal((D,), 0.2, g, F32)).bfloat16()
    ws = moe.alloc_workspace(cfg)
    lws = torch.zeros(moe.moe_linear_w4_workspace_size(T, D, N), dtype=torch.uint8, device="cuda")
    aws = torch.zeros(moe.moe_lora_workspace_size(T, D, N, r, n), dtype=torch.uint8, device="cuda")
    b = {m: torch.zeros((T, D), dtype=BF16, device="cuda") for m in ("sum", "y", "out", "sum2", "y2")}
    logits = torch.zeros((T, N), device="cuda")

    def step():
        moe.moe_block(cfg, gate, d["x"], d["residual"], d["nw"], 1e-6, d["Wg"], d["lb"], d["sb"], d["W13"], None, d["W2"], None, d["W13s"],
                      None, d["W2s"], None, b["sum"], b["y"], b["out"], ws)
        moe.moe_add_rms_norm(T, D, b["out"], b["sum"], w2, 1e-6, b["sum2"], b["y2"])
        moe.moe_linear_w4(T, D, N, 64, b["y2"], qh, sh, None, logits, lws)
        moe.moe_lora(T, D, N, r, n, b["y2"], ld["ids"], ld["A"], ld["B"], ld["scales"], logits, logits, aws)

    step()
    torch.cuda.synchronize()
    want = logits.clone()
    W = moe.dequantize_w4(qh, sh).double()
    base = (b["y2"].double() @ W).float()
    y64, allowed = ref.lora(b["y2"], ld["ids"], ld["A"], ld["B"], ld["scales"], base, F32)
    # base: 512 terms in fp32, weights rounded to bf16 once more by dequantize_w4
    slack = (2.0 ** -8 + 600 * 2 * ref.U) * (b["y2"].double().abs() @ W.abs())
    _within(logits, y64, allowed + slack)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        logits.zero_()
        step()
    s.synchronize()
    assert torch.equal(logits, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    logits.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(logits, want)
    d["x"].copy_(_normal((T, D), 1, g))  # other inputs: nothing is kept from a call
    ld["ids"].copy_(torch.randint(-1, n, (T,), device="cuda", generator=g))
    graph.replay()
    torch.cuda.synchronize()
    got = logits.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(logits, got) and not torch.equal(got, want)


def _three_calls(T, seed):
    """Norm, choice and adapters of T rows: inputs of their own, and a function that runs them in given workspaces."""
    D, E, k, N, r, n = 512, 64, 6, 520, 40, 5
    g, gate, cfg = _gen(seed), moe.make_gate(n_group=8, topk_group=4), moe.make_config(T, 512, 64, 6, 16)
    ld, Wg, sb = _lora_inputs(T, D, N, r, n, F32, seed, "mixed"), _normal((D, E), 0.1, g), _normal((E,), 0.2, g, F32)
    x, res, w = _normal((T, D), 1, g), _normal((T, D), 1, g), _normal((D,), 1, g)
    out = [torch.zeros((T, D), dtype=BF16, device="cuda"), torch.zeros((T, D), dtype=BF16, device="cuda"), torch.zeros((T, E), device="cuda"),
           torch.zeros((T, k), dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda"), torch.zeros((T, N), device="cuda")]

    def run(ws, lws):
        moe.moe_add_rms_norm(T, D, x, res, w, 1e-6, out[0], out[1])
        moe.moe_route_gated(cfg, gate, out[1], Wg, None, sb, out[2], out[3], out[4], ws)
        moe.moe_lora(T, D, N, r, n, out[1], ld["ids"], ld["A"], ld["B"], ld["scales"], ld["base"], out[5], lws)

    return run, out, moe.moe_workspace_size(cfg), moe.moe_lora_workspace_size(T, D, N, r, n)


def _serial(calls):
    """What the calls write, one by one, each waited for."""
    want = []
    for run, out, a, b in calls:
        run(torch.zeros(a, dtype=torch.uint8, device="cuda"), torch.zeros(b, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
        for t in out:
            t.zero_()
    return want


def test_calls_on_two_streams_at_once():
    """Each stream with workspaces of its own, the sizes of one beside those of the other."""
    calls = [_three_calls(T, i) for i, T in enumerate((3000, 7, 64, 1500, 300, 33))]
    want = _serial(calls)
    spaces = [(torch.zeros(max(c[2] for c in calls), dtype=torch.uint8, device="cuda"),
               torch.zeros(max(c[3] for c in calls), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, c in enumerate(calls):
            with torch.cuda.stream(streams[i % 2]):
                c[0](*spaces[i % 2])
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(c[1], w))


def test_graphs_share_workspaces():
    """Captured for several batch sizes in the same workspaces, replayed in any order."""
    calls = [_three_calls(T, i) for i, T in enumerate((1, 16, 65, 2000))]
    want = _serial(calls)
    ws = torch.zeros(max(c[2] for c in calls), dtype=torch.uint8, device="cuda")
    lws = torch.zeros(max(c[3] for c in calls), dtype=torch.uint8, device="cuda")
    graphs = []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c[0](ws, lws)
    for i in (0, 3, 1, 2, 3, 0, 2, 1, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(c[1], w))
