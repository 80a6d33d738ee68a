"""moe_layer_few, moe_linear_w4 and the 4-bit weight conversions on the GPU,
against a plain 64-bit implementation with derived error bounds (_few_ref)."""
import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests import _few_ref as ref
from tests._lib import ensure_library

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp8_e4m3", "fp8_e4m3_nk", "w4_g32", "w4_g64", "w4_g128"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


def _weights(w, lead, K, N, gen):
    """A projection's weights and scales in the layout of `w`, on the GPU."""
    W = torch.empty((*lead, K, N), device="cuda").normal_(0, 0.05, generator=gen)
    if w == "bf16":
        return W.bfloat16(), None
    if w.startswith("w4"):
        return moe.quantize_w4(W, int(w[4:]))
    s = W.abs().amax(-2) / 448
    q = (W / s.unsqueeze(-2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (q if w == "fp8_e4m3" else q.transpose(-1, -2).contiguous()), s


def _inputs(w, T, D, E, k, I, Is, seed=0, bias=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    d = {"x": torch.empty((T, D), device="cuda").normal_(0, 1, generator=g).bfloat16(),
         "Wg": torch.empty((D, E), device="cuda").normal_(0, 0.05, generator=g).bfloat16(),
         "bias": torch.empty(E, device="cuda").normal_(0, 1, generator=g) if bias else None}
    d["W13"], d["s13"] = _weights(w, (E,), D, 2 * I, g)
    d["W2"], d["s2"] = _weights(w, (E,), I, D, g)
    d["W13s"], d["s13s"] = _weights(w, (), D, 2 * Is, g) if Is else (None, None)
    d["W2s"], d["s2s"] = _weights(w, (), Is, D, g) if Is else (None, None)
    return d


def _call(cfg, d, ws, out=None, stream=None):
    if out is None:
        out = torch.full((cfg.T, cfg.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_layer_few(cfg, d["x"], d["Wg"], d["bias"], d["W13"], d["s13"], d["W2"], d["s2"], d["W13s"],
                      d["s13s"], d["W2s"], d["s2s"], out, ws, stream)
    return out


def _check(cfg, d, w, ws, out, act, renorm, rows=None, where="cpu"):
    """out (and the routing left in ws) against the reference; rows: only these."""
    T, E, k = cfg.T, cfg.E, cfg.k
    ids = moe.workspace_view(ws, cfg, "topk_ids", (T, k), torch.int32).long().cpu()
    logits = moe.workspace_view(ws, cfg, "logits", (T, E), torch.float32).double().cpu()
    c = {n: (None if v is None else v.to(where)) for n, v in d.items()}
    ids, logits, out = ids.to(where), logits.to(where), out.to(where)
    if rows is not None:
        c["x"], ids, logits, out = c["x"][rows], ids[rows], logits[rows], out[rows]
    want, tol, exact, el = ref.layer(c["x"], c["Wg"], c["bias"], c["W13"], c["s13"], c["W2"], c["s2"],
                                     c["W13s"], c["s13s"], c["W2s"], c["s2s"], w, k, act, renorm, ids)
    assert ((logits - exact).abs() <= el).all()
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids, order)  # the kernel's own logits, ties to the lower index
    worst = ((out.double() - want).abs() / tol).max().item()
    assert worst <= 1.0, f"{worst} times the allowed error"


SHAPES = [
    # T, D, E, k, I, Is
    (1, 256, 8, 2, 128, 0),
    (1, 640, 7, 3, 384, 128),
    (3, 384, 5, 5, 128, 640),
    (8, 1152, 33, 4, 256, 256),
    (9, 256, 130, 6, 128, 384),
    (17, 512, 16, 1, 128, 128),
    (32, 256, 512, 16, 128, 0),
    (5, 128, 1, 1, 128, 128),
]


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_layer(w, shape):
    T, D, E, k, I, Is = shape
    act, renorm = ("swiglu", True) if T % 2 else ("geglu_tanh", False)
    cfg = moe.make_config(T, D, E, k, I, Is, act, w_dtype=w, renormalize=renorm)
    d = _inputs(w, T, D, E, k, I, Is, seed=T + D, bias=E % 2 == 1)
    ws = moe.alloc_workspace(cfg)
    out = _call(cfg, d, ws)
    assert moe.moe_read_device_status(ws) == 0
    _check(cfg, d, w, ws, out, act, renorm)
    again = _call(cfg, d, ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("w,unit", [("bf16", 8), ("fp8_e4m3", 16), ("fp8_e4m3_nk", 16), ("w4_g32", 32)])
@pytest.mark.parametrize("T,D,I,Is", [(2, 1, 1, 1), (7, 9, 3, 5), (16, 33, 17, 0), (31, 5, 9, 13)])
def test_layer_ragged_widths(w, unit, T, D, I, Is):
    """Widths that are small or odd multiples of the unit: tiles and stages that
    end in the middle."""
    D, I, Is = D * unit, I * unit, Is * unit
    cfg = moe.make_config(T, D, 11, 3, I, Is, w_dtype=w)
    d = _inputs(w, T, D, 11, 3, I, Is, seed=D + I)
    ws = moe.alloc_workspace(cfg)
    out = _call(cfg, d, ws)
    assert moe.moe_read_device_status(ws) == 0
    _check(cfg, d, w, ws, out, "swiglu", True)


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("T", [2, 12, 32])
def test_layer_long_runs(w, T):
    """Every CTA streams more stages than its ring holds, of the shared expert
    (before the routing is known) and of the routed ones; router planes that are
    read by one CTA per token (512 experts)."""
    D, E, k, I, Is = (4096, 512, 2, 128, 2048) if w == "bf16" else (8192, 512, 2, 128, 4096)
    cfg = moe.make_config(T, D, E, k, I, Is, w_dtype=w)
    d = _inputs(w, T, D, E, k, I, Is, seed=T)
    ws = moe.alloc_workspace(cfg)
    out = _call(cfg, d, ws)
    assert moe.moe_read_device_status(ws) == 0
    _check(cfg, d, w, ws, out, "swiglu", True, where="cuda")
    cfg = moe.make_config(T, 2048, 4, 4, 2048, 0, w_dtype=w)
    d = _inputs(w, T, 2048, 4, 4, 2048, 0, seed=T)
    ws = moe.alloc_workspace(cfg)
    out = _call(cfg, d, ws)
    for _ in range(30):  # back to back, nothing waits in between
        again = _call(cfg, d, ws)
    assert torch.equal(out, again)
    assert moe.moe_read_device_status(ws) == 0
    _check(cfg, d, w, ws, out, "swiglu", True, where="cuda")


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("T", [8, 16, 32])
def test_layer_all_tokens_one_expert(w, T):
    """Every token takes expert 5 first (all rows of a pass in one expert)."""
    cfg = moe.make_config(T, 256, 9, 2, 128, 0, w_dtype=w)
    d = _inputs(w, T, 256, 9, 2, 128, 0, seed=T)
    d["bias"] = torch.zeros(9, device="cuda")
    d["bias"][5] = 50.0
    ws = moe.alloc_workspace(cfg)
    out = _call(cfg, d, ws)
    ids = moe.workspace_view(ws, cfg, "topk_ids", (T, 2), torch.int32)
    assert (ids[:, 0] == 5).all()
    _check(cfg, d, w, ws, out, "swiglu", True)


@pytest.mark.parametrize("w", KINDS)
def test_layer_ties_go_to_the_lower_index(w):
    cfg = moe.make_config(4, 256, 24, 6, 128, 0, w_dtype=w)
    d = _inputs(w, 4, 256, 24, 6, 128, 0)
    d["Wg"] = torch.zeros_like(d["Wg"])
    ws = moe.alloc_workspace(cfg)
    out = _call(cfg, d, ws)
    ids = moe.workspace_view(ws, cfg, "topk_ids", (4, 6), torch.int32)
    assert torch.equal(ids.cpu(), torch.arange(6, dtype=torch.int32).expand(4, 6))
    _check(cfg, d, w, ws, out, "swiglu", True)


@pytest.mark.parametrize("w", KINDS)
def test_layer_bad_rows_stay_alone(w):
    """A token with an infinity or NaN flags its logits and leaves the other
    tokens' results as they are; weights of experts nobody chose may be NaN."""
    T = 12
    cfg = moe.make_config(T, 256, 16, 2, 128, 128, w_dtype=w)
    d = _inputs(w, T, 256, 16, 2, 128, 128, seed=3)
    d["bias"] = torch.zeros(16, device="cuda")
    d["bias"][12:] = -1e4  # never chosen
    if w == "bf16":
        d["W13"][12:] = float("nan")
        d["W2"][12:] = float("nan")
    else:
        d["s13"][12:] = float("nan")
        d["s2"][12:] = float("nan")
    ws = moe.alloc_workspace(cfg)
    good = _call(cfg, d, ws)
    assert moe.moe_read_device_status(ws) == 0
    _check(cfg, d, w, ws, good, "swiglu", True)
    d["x"][4, 7] = float("inf")
    d["x"][9, 0] = float("nan")
    bad = _call(cfg, d, ws)
    assert moe.moe_read_device_status(ws) == moe.MOE_DEV_NONFINITE_LOGIT
    rows = [t for t in range(T) if t not in (4, 9)]
    _check(cfg, d, w, ws, bad, "swiglu", True, rows=rows)
    assert torch.isnan(bad[9]).all()
    # the flag is cleared and the next call is clean again
    d["x"][4, 7] = 0.0
    d["x"][9, 0] = 0.0
    _check(cfg, d, w, ws, _call(cfg, d, ws), "swiglu", True)
    assert moe.moe_read_device_status(ws) == 0


def test_layer_zero_tokens_and_zero_x():
    cfg = moe.make_config(3, 256, 8, 2, 128, 128)
    d = _inputs("bf16", 3, 256, 8, 2, 128, 128)
    d["x"].zero_()
    ws = moe.alloc_workspace(cfg)
    assert (_call(cfg, d, ws) == 0).all()
    none = moe.make_config(0, 256, 8, 2, 128, 128)
    keep = torch.ones(3, 256, dtype=torch.bfloat16, device="cuda")
    moe.moe_layer_few(none, d["x"], d["Wg"], None, d["W13"], None, d["W2"], None, d["W13s"], None, d["W2s"],
                      None, keep, ws)
    assert (keep == 1).all()


def test_layer_agrees_with_moe_layer():
    """The same layer by moe_layer: both are within the bound of the exact one,
    so they differ by at most two of them."""
    T, D, E, k, I, Is = 16, 512, 64, 4, 256, 256
    cfg = moe.make_config(T, D, E, k, I, Is)
    d = _inputs("bf16", T, D, E, k, I, Is, seed=9)
    ws = moe.alloc_workspace(cfg)
    few = _call(cfg, d, ws)
    full = torch.empty_like(few)
    moe.moe_layer(cfg, d["x"], d["Wg"], None, d["W13"], None, d["W2"], None, d["W13s"], None, d["W2s"], None,
                  full, ws)
    _check(cfg, d, "bf16", ws, few, "swiglu", True)
    _check(cfg, d, "bf16", ws, full, "swiglu", True)
    assert torch.equal(few, _call(cfg, d, ws))  # moe_layer in between leaves the workspace usable


def test_layer_prefill_then_decode_in_4_bits():
    """Weights kept in 4 bits: a prompt through moe_layer on dequantised weights,
    then single tokens through moe_layer_few on the codes, on one stream."""
    D, E, k, I = 256, 16, 2, 128
    d = _inputs("w4_g64", 40, D, E, k, I, 0, seed=4)
    W13, W2 = moe.dequantize_w4(d["W13"], d["s13"]), moe.dequantize_w4(d["W2"], d["s2"])
    big = moe.make_config(40, D, E, k, I)
    ws = moe.alloc_workspace(big)
    prompt = torch.empty((40, D), dtype=torch.bfloat16, device="cuda")
    moe.moe_layer(big, d["x"], d["Wg"], None, W13, None, W2, None, None, None, None, None, prompt, ws)
    one = moe.make_config(1, D, E, k, I, w_dtype="w4_g64")
    ws1 = moe.alloc_workspace(one)
    for t in (0, 17, 39):
        dt = dict(d, x=d["x"][t:t + 1].contiguous())
        out = _call(one, dt, ws1)
        _check(one, dt, "w4_g64", ws1, out, "swiglu", True)
    _check(big, dict(d, W13=W13, s13=None, W2=W2, s2=None), "bf16", ws, prompt, "swiglu", True)


@pytest.mark.parametrize("w", ["bf16", "fp8_e4m3_nk", "w4_g128"])
def test_layer_graph_streams_and_shared_workspace(w):
    """Two captured layers of different sizes share one workspace, replayed in
    turn; eager calls on two streams with a workspace each."""
    a = (8, 512, 32, 4, 256, 128)
    b = (1, 256, 16, 2, 128, 0)
    runs = []
    cfgs = [moe.make_config(*s, w_dtype=w) for s in (a, b)]
    ws = torch.zeros(max(moe.moe_workspace_size(c) for c in cfgs), dtype=torch.uint8, device="cuda")
    for s, cfg in zip((a, b), cfgs):
        d = _inputs(w, *s, seed=s[0])
        out = torch.empty((cfg.T, cfg.D), dtype=torch.bfloat16, device="cuda")
        want = _call(cfg, d, moe.alloc_workspace(cfg))
        _call(cfg, d, ws, out)
        runs.append([cfg, d, out, want, None])
    st = torch.cuda.Stream()
    for r in runs:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            _call(r[0], r[1], ws, r[2])
        r[4] = g
    for _ in range(3):
        for r in runs:
            r[2].fill_(7.0)
            r[4].replay()
        torch.cuda.synchronize()
        for r in runs:
            assert torch.equal(r[2], r[3])
    # new inputs in the captured buffers
    runs[0][1]["x"].copy_(runs[0][1]["x"].flip(0))
    runs[0][4].replay()
    torch.cuda.synchronize()
    assert torch.equal(runs[0][2], runs[0][3].flip(0))
    # two streams, a workspace each
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [moe.alloc_workspace(c) for c in cfgs]
    torch.cuda.synchronize()
    for _ in range(4):
        for r, s, wk in zip(runs, streams, wss):
            _call(r[0], r[1], wk, r[2], s)
    torch.cuda.synchronize()
    assert torch.equal(runs[0][2], runs[0][3].flip(0)) and torch.equal(runs[1][2], runs[1][3])


# ------------------------------------------------------------------ linear
def _w4(N, K, g, zeros, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (torch.rand((N, K // g), device="cuda", generator=gen) * 0.02 + 0.001).bfloat16()
    z = torch.randint(0, 256, (N, K // g), dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return q, s, z


def _linear_ws(M, K, N):
    return torch.zeros(moe.moe_linear_w4_workspace_size(M, K, N), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("M,K,N", [(1, 128, 1), (1, 384, 127), (2, 256, 128), (8, 640, 129), (9, 2816, 1000),
                                   (16, 128, 300), (17, 1152, 257), (32, 4096, 515), (5, 16384, 40)])
@pytest.mark.parametrize("zeros", [False, True])
def test_linear(g, M, K, N, zeros):
    q, s, z = _w4(N, K, g, zeros, seed=M + K + N)
    x = torch.randn(M, K, device="cuda").bfloat16()
    ws = _linear_ws(M, K, N)
    for dt in (torch.bfloat16, torch.float32):
        y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
        moe.moe_linear_w4(M, K, N, g, x, q, s, z, y, ws)
        want, tol = ref.linear(x.cpu(), q.cpu(), s.cpu(), None if z is None else z.cpu(), dt)
        worst = ((y.double().cpu() - want).abs() / tol).max().item()
        assert worst <= 1.0, f"{worst} times the allowed error"
        again = torch.empty_like(y)
        moe.moe_linear_w4(M, K, N, g, x, q, s, z, again, ws)
        assert torch.equal(y, again)
    assert moe.moe_read_device_status(ws) == 0


def test_linear_smallest_group_and_k():
    for g in (32, 64, 128):
        q, s, z = _w4(3, g, g, True)
        x = torch.randn(1, g, device="cuda").bfloat16()
        y = torch.empty(1, 3, device="cuda")
        moe.moe_linear_w4(1, g, 3, g, x, q, s, z, y, _linear_ws(1, g, 3))
        want, tol = ref.linear(x.cpu(), q.cpu(), s.cpu(), z.cpu(), torch.float32)
        assert ((y.double().cpu() - want).abs() <= tol).all()


def test_linear_nonfinite_rows_stay_alone():
    M, K, N, g = 11, 512, 200, 64
    q, s, z = _w4(N, K, g, True)
    x = torch.randn(M, K, device="cuda").bfloat16()
    ws = _linear_ws(M, K, N)
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_w4(M, K, N, g, x, q, s, z, y, ws)
    x[3, 5] = float("nan")
    x[8, 100] = float("inf")
    y2 = torch.empty_like(y)
    moe.moe_linear_w4(M, K, N, g, x, q, s, z, y2, ws)
    rows = [m for m in range(M) if m not in (3, 8)]
    assert torch.equal(y[rows], y2[rows])
    assert torch.isnan(y2[3]).all() and not torch.isfinite(y2[8]).any()


def test_linear_workspace_serves_other_sizes_graphs_and_streams():
    """One workspace for products of several sizes in a row, eager and captured."""
    sizes = [(1, 4096, 700, 128), (32, 256, 4000, 32), (9, 8192, 130, 64)]
    ws = torch.zeros(max(moe.moe_linear_w4_workspace_size(*s[:3]) for s in sizes), dtype=torch.uint8,
                     device="cuda")
    jobs = []
    for M, K, N, g in sizes:
        q, s, z = _w4(N, K, g, False, seed=N)
        x = torch.randn(M, K, device="cuda").bfloat16()
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        args = (M, K, N, g, x, q, s, z, y)
        moe.moe_linear_w4(*args, _linear_ws(M, K, N))
        jobs.append((args, y.clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for args, _ in jobs:
            moe.moe_linear_w4(*args, ws)
    for _ in range(3):
        for args, want in jobs:
            args[-1].zero_()
            moe.moe_linear_w4(*args, ws)
            assert torch.equal(args[-1], want)
            args[-1].zero_()
        graph.replay()
        for args, want in jobs:
            assert torch.equal(args[-1], want)


# ------------------------------------------------------ 4-bit weight conversions
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,K,N,g", [(1, 32, 1, 32), (3, 128, 65, 64), (2, 256, 129, 128), (1, 640, 64, 32)])
def test_quantize_round_trip(dt, G, K, N, g):
    W = (torch.randn(G, K, N, device="cuda") * 0.1).to(dt)
    W[0, :g, 0] = 0
    q, s = moe.quantize_w4(W, g)
    wt = W.float().transpose(1, 2).reshape(G, N, K // g, g)
    amax = wt.abs().amax(-1)
    # division by seven and the codes' division are IEEE single precision on both sides
    want_s = torch.where(amax > 0, (amax / 7.0).bfloat16().float(), torch.ones_like(amax))
    assert torch.equal(s.float(), want_s)
    codes = (torch.round(wt / want_s[..., None]).clamp(-8, 7) + 8).to(torch.uint8).reshape(G, N, K)
    assert torch.equal(q, codes[..., 0::2] | (codes[..., 1::2] << 4))
    back = moe.dequantize_w4(q, s)
    want = ref.unpack_w4(q, s).transpose(1, 2).float().bfloat16()
    assert torch.equal(back, want)
    # the largest value is at most 7 (1 + 2^-8) steps, so clamping takes nothing off
    step = want_s.repeat_interleave(g, -1).transpose(1, 2)
    assert ((back.float() - W.float()).abs() <= step * (0.5 + 2 ** -6) + 2.0 ** -8 * back.float().abs()).all()
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, device="cuda")
    assert torch.equal(moe.dequantize_w4(q, s, z), ref.unpack_w4(q, s, z).transpose(1, 2).float().bfloat16())
    one = moe.quantize_w4(W[0], g)
    assert torch.equal(one[0], q[0]) and torch.equal(one[1], s[0])
    assert torch.equal(moe.dequantize_w4(*one), back[0])


def test_quantize_nonfinite_group_is_nan():
    W = torch.randn(64, 8, device="cuda")
    W[3, 2] = float("inf")
    W[40, 5] = float("nan")
    back = moe.dequantize_w4(*moe.quantize_w4(W, 32))
    bad = torch.isnan(back)
    want = torch.zeros_like(bad)
    want[:32, 2] = True
    want[32:, 5] = True
    assert torch.equal(bad, want)


def _check_some_columns(M, K, N, g, zeros, dt, offset=0):
    """A large product against 64 bits at 300 of its columns, both ends among them."""
    q, s, z = _w4(N, K, g, zeros, seed=M + N)
    if zeros and offset:  # zero points need no alignment
        raw = torch.empty(z.numel() + offset, dtype=torch.uint8, device="cuda")
        raw[offset:].copy_(z.reshape(-1))
        z = raw[offset:].view_as(z)
    x = torch.randn(M, K, device="cuda").bfloat16()
    ws = _linear_ws(M, K, N)
    y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    moe.moe_linear_w4(M, K, N, g, x, q, s, z, y, ws)
    gen = torch.Generator().manual_seed(3)
    cols = torch.cat([torch.arange(20), torch.arange(N - 20, N), torch.randint(0, N, (260,), generator=gen)])
    at = cols.cuda()
    want, tol = ref.linear(x.cpu(), q[at].cpu(), s[at].cpu(), None if z is None else z[at].cpu(), dt)
    worst = ((y[:, at].double().cpu() - want).abs() / tol).max().item()
    assert worst <= 1.0, f"{worst} times the allowed error"
    assert torch.isfinite(y).all() and moe.moe_read_device_status(ws) == 0
    again = torch.empty_like(y)
    moe.moe_linear_w4(M, K, N, g, x, q, s, z, again, ws)
    assert torch.equal(y, again)


@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("M,K,N,zeros,dt", [
    (9, 8192, 8200, True, torch.bfloat16),      # 9 to 16 rows, weights of many stages
    (16, 384, 131071, False, torch.float32),
    (32, 256, 117001, True, torch.float32),     # strips of one stage
    (17, 2816, 40000, False, torch.bfloat16),   # groups of a row no multiple of eight
    (31, 640, 70002, True, torch.bfloat16),
])
def test_linear_many_strips(M, K, N, g, zeros, dt):
    _check_some_columns(M, K, N, g, zeros, dt)


@pytest.mark.parametrize("M,N", [(3, 300), (11, 700), (20, 700)])
def test_linear_unaligned_zero_points(M, N):
    for offset in (1, 2, 4):
        _check_some_columns(M, 2048, N, 64, True, torch.float32, offset)


def test_linear_nonfinite_rows_stay_alone_with_many_rows():
    M, K, N, g = 29, 1024, 600, 32
    q, s, z = _w4(N, K, g, True)
    x = torch.randn(M, K, device="cuda").bfloat16()
    ws = _linear_ws(M, K, N)
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_w4(M, K, N, g, x, q, s, z, y, ws)
    x[3, 5] = float("nan")
    x[28, 1000] = float("-inf")
    y2 = torch.empty_like(y)
    moe.moe_linear_w4(M, K, N, g, x, q, s, z, y2, ws)
    rows = [m for m in range(M) if m not in (3, 28)]
    assert torch.equal(y[rows], y2[rows])
    assert torch.isnan(y2[3]).all() and not torch.isfinite(y2[28]).any()


@pytest.mark.parametrize("w", ["w4_g32", "w4_g64"])
@pytest.mark.parametrize("T,D,E,k,I,Is", [
    (19, 4096, 64, 8, 704, 2112),   # long strips of the shared expert, then short ones
    (20, 4096, 32, 4, 1536, 320),   # short ones first
    (3, 8192, 16, 2, 2048, 64),
    (32, 6144, 48, 3, 256, 704),    # both short, of one and of three stages
    (1, 8192, 8, 8, 576, 0),
])
def test_layer_strips_of_two_lengths(w, T, D, E, k, I, Is):
    cfg = moe.make_config(T, D, E, k, I, Is, w_dtype=w)
    d = _inputs(w, T, D, E, k, I, Is, seed=I)
    ws = moe.alloc_workspace(cfg)
    out = _call(cfg, d, ws)
    for _ in range(10):
        again = _call(cfg, d, ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert moe.moe_read_device_status(ws) == 0
    _check(cfg, d, w, ws, out, "swiglu", True, where="cuda")


def test_calls_on_several_streams_at_once():
    """Products of many and of few rows and whole layers side by side, each stream
    with a workspace of its own; a workspace goes from stream to stream in order."""
    jobs = []
    for M, K, N, g in ((32, 2048, 20000, 64), (20, 4096, 9000, 32), (3, 2048, 9000, 128)):
        q, s, z = _w4(N, K, g, True, seed=M)
        x = torch.randn(M, K, device="cuda").bfloat16()
        y = torch.empty(M, N, device="cuda")
        args = (M, K, N, g, x, q, s, z, y, _linear_ws(M, K, N))
        moe.moe_linear_w4(*args)
        jobs.append((lambda st, a=args: moe.moe_linear_w4(*a, stream=st), y, y.clone()))
    cfg = moe.make_config(12, 1024, 16, 4, 768, 256, w_dtype="w4_g64")
    d = _inputs("w4_g64", 12, 1024, 16, 4, 768, 256, seed=5)
    ws, out = moe.alloc_workspace(cfg), torch.empty(12, 1024, dtype=torch.bfloat16, device="cuda")
    _call(cfg, d, ws, out)
    jobs.append((lambda st: _call(cfg, d, ws, out, st), out, out.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for turn in range(4):
        for _, y, _ in jobs:
            y.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for i, (run, _, _) in enumerate(jobs):
                run(streams[(i + turn) % len(streams)])
        torch.cuda.synchronize()
        for _, y, want in jobs:
            assert torch.equal(y, want)
    assert moe.moe_read_device_status(ws) == 0
