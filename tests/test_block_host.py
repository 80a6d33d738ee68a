"""Host-side checks of moe_add_rms_norm, moe_route_gated, moe_lora and moe_block:
everything refused here is refused before any CUDA call."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests import _block_ref as ref
from tests._lib import ensure_library

P = 1 << 20  # a fake, aligned device address: validation fails before any use
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5


@pytest.fixture(scope="module")
def lib():
    return ensure_library()


# ------------------------------------------------------------------- norm
Q = 1 << 21  # another


def _norm(lib, rows=4, D=256, dt=moe.MOE_BF16, x=P, res=P, w=P, eps=1e-6, sum_out=P, y=Q, q=P, group=0, s=P):
    return lib.moe_add_rms_norm(rows, D, dt, x, res, w, eps, sum_out, y, q, group, s, None)


def test_norm_refusals(lib):
    assert _norm(lib, rows=0) == 0
    assert _norm(lib, rows=0, x=None, res=None, w=None, sum_out=None, y=None, q=None, s=None) == 0
    for bad in ({"rows": -1}, {"D": 0}, {"D": 252}, {"eps": -1e-6}, {"eps": math.inf}, {"eps": math.nan}, {"group": 16},
                {"group": 256}, {"D": 264, "group": 32}, {"x": None}, {"w": None}, {"y": None, "q": None, "s": None},
                {"s": None}, {"q": None}, {"y": P}, {"x": P + 8}, {"res": P + 2}, {"w": P + 4}, {"sum_out": P + 8}, {"y": P + 8},
                {"q": P + 4}, {"s": P + 4}):
        assert _norm(lib, **bad) == INVALID, bad
    for bad in ({"dt": moe.MOE_FP8_E4M3}, {"dt": -1}, {"D": 32776}):
        assert _norm(lib, **bad) == UNSUPPORTED, bad


def test_norm_wrapper_compares_its_tensors():
    T, D = 3, 256
    x = torch.zeros(T, D, dtype=torch.bfloat16)
    good = dict(x=x, residual=x, weight=x[0], sum_out=x, y=x, q=torch.zeros(T, D, dtype=torch.uint8),
                q_scales=torch.zeros(T, D // 64))

    def call(**other):
        a = dict(good, **other)
        moe.moe_add_rms_norm(T, D, a["x"], a["residual"], a["weight"], 1e-6, a["sum_out"], a["y"], a["q"], a["q_scales"], 64)

    ensure_library()
    for a in ({}, {"residual": None}, {"sum_out": None}, {"y": None}, {"q": torch.zeros(T, D).to(torch.float8_e4m3fn)}):
        with pytest.raises(ValueError, match="CUDA device"):
            call(**a)
    for name, t in good.items():
        with pytest.raises(ValueError, match="moe_add_rms_norm takes"):
            call(**{name: t[:-1].contiguous()})
        with pytest.raises(ValueError, match="moe_add_rms_norm takes"):
            call(**{name: t.double()})


# ------------------------------------------------------------------- gate
def _cfg(T=4, E=64, k=4, **kw):
    return moe.make_config(T, 256, E, k, 128, **kw)


def _route(lib, cfg, gate, x=P, Wg=P, lb=None, sb=P, logits=P, ids=P, w=P, ws=P, n=None):
    return lib.moe_route_gated(ctypes.byref(cfg), None if gate is None else ctypes.byref(gate), x, Wg, lb, sb, logits, ids,
                               w, ws, moe.moe_workspace_size(cfg) if n is None else n, None)


BAD_GATES = [dict(n_group=0), dict(n_group=3), dict(n_group=64), dict(n_group=4, topk_group=0), dict(n_group=4, topk_group=5),
             dict(n_group=32, topk_group=1), dict(scale=math.inf), dict(scale=math.nan)]


def test_gate_refusals(lib):
    assert _route(lib, _cfg(T=0), moe.make_gate()) == 0
    assert _route(lib, _cfg(), None) == INVALID
    for bad in BAD_GATES:
        assert _route(lib, _cfg(), moe.make_gate(**bad)) == INVALID, bad
    for field in ("score", "group_score"):
        for v in (-1, 2):
            g = moe.make_gate()
            setattr(g, field, v)
            assert _route(lib, _cfg(), g) == INVALID
    g = moe.make_gate(n_group=8, topk_group=2)
    for bad in ({"Wg": None}, {"x": P + 8}, {"Wg": P + 8}, {"x": None, "lb": P}, {"logits": None}, {"ids": None}, {"w": None}):
        assert _route(lib, _cfg(), g, **bad) == INVALID, bad
    assert _route(lib, _cfg(E=60), moe.make_gate(n_group=4, topk_group=1)) == INVALID  # rows of W_g
    assert _route(lib, _cfg(), g, ws=None) == WORKSPACE
    assert _route(lib, _cfg(), g, n=1000) == WORKSPACE
    with pytest.raises(KeyError):
        moe.make_gate("tanh")


def test_gate_wrapper_compares_its_tensors(lib):
    T, E, k, D = 3, 64, 4, 256
    cfg = _cfg(T=T)
    good = dict(x=torch.zeros(T, D).bfloat16(), Wg=torch.zeros(D, E).bfloat16(), lb=torch.zeros(E), sb=torch.zeros(E),
                logits=torch.zeros(T, E), ids=torch.zeros(T, k, dtype=torch.int32), w=torch.zeros(T, k))
    ws = torch.zeros(moe.moe_workspace_size(cfg), dtype=torch.uint8)

    def call(**other):
        a = dict(good, **other)
        moe.moe_route_gated(cfg, moe.make_gate(), a["x"], a["Wg"], a["lb"], a["sb"], a["logits"], a["ids"], a["w"], ws)

    for a in ({}, {"x": None, "Wg": None, "lb": None}, {"sb": None}):
        with pytest.raises(ValueError, match="CUDA device"):
            call(**a)
    for name, t in good.items():
        for bad in (t[:-1].contiguous(), t.double()):
            with pytest.raises(ValueError, match="moe_route_gated takes"):
                call(**{name: bad})


# ------------------------------------------------------------------- lora
def _lora(lib, T=4, K=256, N=64, r=16, n=3, x=P, ids=P, A=P, B=P, s=P, base=P, y=P, dt=moe.MOE_BF16, ws=P, size=1 << 40):
    return lib.moe_lora(T, K, N, r, n, x, ids, A, B, s, base, y, dt, ws, size, None)


def test_lora_refusals(lib):
    for n in (1, 2, 16384):
        assert _lora(lib, T=0, n=n) == 0
        for T in (0, 1, 64, 65, 1 << 30):
            assert moe.moe_lora_workspace_size(T, 1 << 24, 8, 256, n) > 0
    assert _lora(lib, T=0, x=None, ids=None, y=None, base=None) == 0
    for bad in ({"T": -1}, {"T": (1 << 30) + 1}, {"K": 0}, {"K": 252}, {"N": 12}, {"N": -8}, {"r": 0}, {"r": 12}, {"n": 0}, {"K": (1 << 24) + 8},
                {"N": (1 << 24) + 8}, {"x": None}, {"ids": None}, {"A": None}, {"B": None}, {"y": None}, {"x": P + 8},
                {"A": P + 2}, {"B": P + 8}, {"y": P + 8}, {"base": P + 8}, {"ids": P + 2}, {"s": P + 1}):
        assert _lora(lib, **bad) == INVALID, bad
    for bad in ({"r": 264}, {"n": 16385}, {"dt": moe.MOE_FP8_E4M3}, {"dt": -1}):
        assert _lora(lib, **bad) == UNSUPPORTED, bad
    need = moe.moe_lora_workspace_size(4, 256, 64, 16, 3)
    assert need > 0
    for bad in ({"ws": None}, {"ws": P + 16}, {"size": need - 1}):
        assert _lora(lib, **bad) == WORKSPACE, bad
    for bad in ((-1, 256, 64, 16, 3), (4, 250, 64, 16, 3), (4, 256, 64, 264, 3), (4, 256, 64, 16, 0)):
        assert moe.moe_lora_workspace_size(*bad) == 0


def test_lora_does_not_write_its_input(lib):
    assert _lora(lib, K=64, N=64, x=P, y=P, base=P) == INVALID  # rows would be read after they are written
    assert _lora(lib, T=0, K=64, N=64, x=P, y=P, base=P) == 0
    for bad in ({"x": None}, {"ids": None}, {"A": None}, {"B": None}, {"y": None}, {"x": P + 8}, {"A": P + 2}, {"B": P + 8},
                {"y": Q + 8}, {"base": P + 8}, {"ids": P + 2}, {"s": P + 1}):  # refused with a y of its own too
        assert _lora(lib, **{"y": Q, **bad}) == INVALID, bad


def test_lora_wrapper_compares_its_tensors(lib):
    T, K, N, r, n = 3, 64, 24, 8, 2
    good = dict(x=torch.zeros(T, K).bfloat16(), ids=torch.zeros(T, dtype=torch.int32), A=torch.zeros(n, r, K).bfloat16(),
                B=torch.zeros(n, N, r).bfloat16(), scales=torch.zeros(n), base=torch.zeros(T, N), y=torch.zeros(T, N))
    ws = torch.zeros(moe.moe_lora_workspace_size(T, K, N, r, n), dtype=torch.uint8)

    def call(**other):
        a = dict(good, **other)
        moe.moe_lora(T, K, N, r, n, a["x"], a["ids"], a["A"], a["B"], a["scales"], a["base"], a["y"], ws)

    for a in ({}, {"scales": None}, {"base": None}, {"y": good["y"].bfloat16(), "base": good["y"].bfloat16()}):
        with pytest.raises(ValueError, match="CUDA device"):
            call(**a)
    for name, t in good.items():
        with pytest.raises(ValueError, match="moe_lora takes"):
            call(**{name: t[:-1].contiguous()})
        with pytest.raises((ValueError, moe.MoEError)):
            call(**{name: t.double()})
    with pytest.raises(ValueError, match="moe_lora takes"):
        call(y=good["y"].bfloat16())  # a base of another type


# ------------------------------------------------------------------ block
def _block(lib, cfg, gate=None, x=P, res=None, nw=P, eps=1e-6, sb=None, W13=P, s13=None, sum_out=None, y=Q, out=P, ws=P, n=None):
    return lib.moe_block(ctypes.byref(cfg), None if gate is None else ctypes.byref(gate), x, res, nw, eps, P, None, sb, W13, s13,
                         P, s13, None, None, None, None, sum_out, y, out, ws, moe.moe_workspace_size(cfg) if n is None else n, None)


def test_block_refusals(lib):
    assert _block(lib, _cfg(T=0)) == 0
    assert _block(lib, _cfg(T=0), nw=None, y=None, eps=0.0) == 0
    for bad in ({"x": None}, {"x": P + 8}, {"W13": None}, {"out": None}, {"s13": P}, {"y": None}, {"y": P}, {"y": P + 8}, {"res": Q}, {"sum_out": Q}, {"nw": P + 8},
                {"res": P + 8}, {"sum_out": P + 8}, {"eps": -1.0}, {"eps": math.nan}, {"sb": P},
                {"nw": None}, {"nw": None, "y": None}, {"nw": None, "y": None, "eps": 0.0, "res": P},
                {"nw": None, "y": None, "eps": 0.0, "sum_out": P}):
        assert _block(lib, _cfg(), **bad) == INVALID, bad
    for bad in BAD_GATES:
        assert _block(lib, _cfg(), moe.make_gate(**bad)) == INVALID, bad
    w4 = dict(w_dtype="w4_g64")
    assert _block(lib, _cfg(T=33, **w4), s13=P) == UNSUPPORTED  # 4-bit weights: a few tokens
    assert _block(lib, _cfg(T=0, **w4), s13=P) == 0
    for c in (w4, dict(w_dtype="fp8_e4m3")):
        assert _block(lib, _cfg(T=4, **c)) == INVALID  # no scales
        assert _block(lib, _cfg(T=4, **c), s13=P + 8) == INVALID
    assert _block(lib, _cfg(T=4), n=moe.moe_workspace_size(_cfg(T=4)) - 1) == WORKSPACE
    assert _block(lib, moe.make_config(4, 32776, 64, 4, 128)) == UNSUPPORTED
    assert _block(lib, _cfg(), n=1000) == WORKSPACE


def test_block_outputs_are_three_buffers(lib):
    R = 1 << 22
    for bad in ({"y": Q, "out": Q}, {"sum_out": R, "out": R}):
        assert _block(lib, _cfg(), **bad) == INVALID, bad
    assert _block(lib, _cfg(T=0), y=Q, out=R, sum_out=P) == 0


def test_block_wrapper_compares_its_tensors(lib):
    T, D, E = 3, 256, 64
    cfg = _cfg(T=T)
    x, W = torch.zeros(T, D).bfloat16(), torch.zeros(8).bfloat16()
    good = dict(x=x, residual=x, nw=x[0], Wg=torch.zeros(D, E).bfloat16(), lb=torch.zeros(E), sb=torch.zeros(E), sum_out=x, y=x, out=x)

    def call(**other):
        a = dict(good, **other)
        moe.moe_block(cfg, moe.make_gate(), a["x"], a["residual"], a["nw"], 1e-6, a["Wg"], a["lb"], a["sb"], W, None, W, None, None, None,
                      None, None, a["sum_out"], a["y"], a["out"], W)

    for a in ({}, {"residual": None, "sum_out": None}, {"sb": None, "lb": None}):
        with pytest.raises(ValueError, match="CUDA device"):
            call(**a)
    for name, t in good.items():
        for bad in (t[:-1].contiguous(), t.double()):
            with pytest.raises(ValueError, match="moe_block takes"):
                call(**{name: bad})


# ------------------------------------------------------------------- call
def test_call_gives_the_calls_their_arguments(lib):
    """The same refusals, one argument wrong at a time, from the words as from the arguments."""
    need = moe.moe_lora_workspace_size(4, 256, 64, 16, 3)
    good = [0, 256, 64, 16, 3, P, P, P, P, P, P, P, moe.MOE_BF16, P, need, 0]
    for i, bad, want in [(0, 0, 0), (0, -1, -1), (1, 12, -1), (2, 4, -1), (3, 264, -2), (4, 0, -1), (12, 9, -2), (13, P + 8, -5), (14, need - 1, -5)]:
        a = list(good)
        a[i] = bad
        if i == 14:
            a[0] = 4
        assert lib.moe_call(moe._LORA, moe._LORA_WORDS(*a)) == want == lib.moe_lora(*a)
    for i in (5, 6, 7, 8, 11):
        a = [4] + good[1:]
        a[i] = 0
        assert lib.moe_call(moe._LORA, moe._LORA_WORDS(*a)) == -1
    good = [0, 256, moe.MOE_BF16, P, P, P, 1e-6, P, Q, P, 0, P, 0]
    for i, bad, want in [(0, 0, 0), (1, 12, -1), (2, 9, -2), (6, -1.0, -1), (6, math.inf, -1), (10, 16, -1)]:
        a = list(good)
        a[i] = bad
        assert lib.moe_call(moe._NORM, moe._NORM_WORDS(*a)) == want == lib.moe_add_rms_norm(*a)
    for i in (3, 5, 9, 11):
        a = [4] + good[1:]
        a[i] = 0
        assert lib.moe_call(moe._NORM, moe._NORM_WORDS(*a)) == -1
    cfg, gate = _cfg(), moe.make_gate()
    n = moe.moe_workspace_size(cfg)
    good = [ctypes.addressof(cfg), ctypes.addressof(gate), P, P, 0, P, P, P, P, P, n, 0]
    for i, bad, want in [(0, 0, -1), (1, 0, -1), (2, P + 8, -1), (3, 0, -1), (6, 0, -1), (7, 0, -1), (8, 0, -1), (9, 0, -5), (10, 100, -5)]:
        a = list(good)
        a[i] = bad
        assert lib.moe_call(moe._ROUTE_GATED, moe._ROUTE_GATED_WORDS(*a)) == want
    assert lib.moe_call(3, moe._LORA_WORDS(*range(16))) == -1 and lib.moe_call(0, None) == -1


def test_call_takes_no_integer_of_more_than_32_bits(lib):
    lora = [0, 256, 64, 16, 3, P, P, P, P, P, P, Q, moe.MOE_BF16, P, 1 << 40, 0]
    norm = [0, 256, moe.MOE_BF16, P, P, P, 1e-6, P, Q, P, 0, P, 0]
    for call, words, good, places in ((moe._LORA, moe._LORA_WORDS, lora, (0, 1, 2, 3, 4, 12)),
                                      (moe._NORM, moe._NORM_WORDS, norm, (0, 1, 2, 10))):
        assert lib.moe_call(call, words(*good)) == 0
        for i in places:
            for add in (1 << 32, -1 << 32, 1 << 40):
                a = list(good)
                a[i] += add
                assert lib.moe_call(call, words(*a)) == INVALID, (call, i)


# -------------------------------------------------------------- reference
def test_gate_reference_on_hand_written_rows():
    l = torch.tensor([[0.0, 2.0, 2.0, -1.0, 3.0, float("nan"), 1.0, 1.0]])
    ids, w, _ = ref.gate(l, None, 3, renorm=False)
    assert ids.tolist() == [[4, 1, 2]] and abs(w[0, 0] - 1 / (1 + math.exp(-3))) < 1e-15
    # groups of two: sums of sigmoids (.5 + .88), (.88 + .27), (.95), (.73 + .73)
    ids, _, _ = ref.gate(l, None, 2, n_group=4, topk_group=2)
    assert ids.tolist() == [[1, 6]]
    ids, _, _ = ref.gate(l, None, 2, n_group=4, topk_group=2, group_score="max")
    assert ids.tolist() == [[4, 1]]
    ids, w, _ = ref.gate(l, torch.tensor([9.0, 0, 0, 0, 0, 9.0, 0, 0]), 2, score="softmax", scale=2.0)
    assert ids.tolist() == [[0, 4]] and abs(w[0].sum() - 2.0) < 1e-12 and abs(w[0, 1] / w[0, 0] - math.exp(3)) < 1e-9
