"""moe_layer_few and moe_linear_w4 on the GPU where something has gone wrong
before or around them."""
import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests import _few_tight as tight
from tests._few_ref import unpack_w4
from tests._lib import ensure_library
from tests.test_gpu_few import _call, _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


@pytest.mark.parametrize("w", ["bf16", "w4_g64"])
@pytest.mark.parametrize("left_over", ["one short", "many"])
def test_layer_survives_a_barrier_that_gives_up(w, left_over):
    """Arrivals left over at the barrier before the chosen experts are read (which
    moe.h says to clear): CTAs go on with whatever the workspace holds, or wait until
    they give up (2 s).  The status says so, nothing outside the workspace is
    written, and a cleared workspace serves the next call."""
    T, D, E, k, I = 5, 2048, 512, 10, 128
    cfg = moe.make_config(T, D, E, k, I, w_dtype=w)
    d = _inputs(w, T, D, E, k, I, 0, seed=2)
    n, guard = moe.moe_workspace_size(cfg), 1 << 20
    room = torch.zeros(n + guard, dtype=torch.uint8, device="cuda")
    room[n:] = 0xA5
    ws = room[:n]
    want = _call(cfg, d, ws).clone()
    assert moe.moe_read_device_status(ws) == 0
    moe.workspace_view(ws, cfg, "topk_ids", (T, k), torch.int32).fill_(3)  # one expert, ten times a token
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws[:256].view(torch.int32)[32 + 8] = sms - 1 if left_over == "one short" else 1 << 20
    _call(cfg, d, ws)
    assert moe.moe_read_device_status(ws) & moe.MOE_DEV_WAIT_TIMEOUT
    assert (room[n:] == 0xA5).all()
    ws[:256].zero_()
    out = _call(cfg, d, ws)
    assert torch.equal(out, want) and moe.moe_read_device_status(ws) == 0
    _check(cfg, d, w, ws, out, "swiglu", True)


def test_moe_layer_for_few_tokens_in_a_larger_batch_s_workspace():
    """moe_layer for 16 tokens in a workspace for 64, which moe_layer_few's scratch
    does not fit into."""
    D, E, k, I = 2048, 128, 8, 768
    cfg = moe.make_config(16, D, E, k, I)
    n, guard = moe.moe_workspace_size(moe.make_config(64, D, E, k, I)), 1 << 16
    assert n < moe.moe_workspace_size(cfg)
    room = torch.zeros(n + guard, dtype=torch.uint8, device="cuda")
    room[n:] = 0xA5
    d = _inputs("bf16", 16, D, E, k, I, 0, seed=6)
    out = torch.full((16, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    args = [d[i] for i in ("x", "Wg", "bias", "W13", "s13", "W2", "s2", "W13s", "s13s", "W2s", "s2s")]
    moe.moe_layer(cfg, *args, out, room[:n])
    assert moe.moe_read_device_status(room) == 0
    _check(cfg, d, "bf16", room[:n], out, "swiglu", True, where="cuda")
    assert (room[n:] == 0xA5).all()
    with pytest.raises(moe.MoEError):
        _call(cfg, d, room[:n], out)


def test_linear_of_no_rows():
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(8, 64, dtype=torch.uint8, device="cuda")
    s = torch.zeros(8, 2, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(moe.moe_linear_w4_workspace_size(0, 128, 8), dtype=torch.uint8, device="cuda")
    moe.moe_linear_w4(0, 128, 8, 64, x, q, s, None, torch.empty(0, 8, device="cuda"), ws)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("M,K,N,g,zeros", [
    (1, 65536, 140001, 128, True),   # 4.6 GB of codes
    (20, 65536, 140001, 64, False),  # the kernel for many rows
    (3, 16384, 1000, 32, True),
    (32, 16384, 1000, 32, True),
])
def test_linear_long_sums_and_offsets_past_32_bits(M, K, N, g, zeros):
    """Some columns, the last ones among them, within the size of a sum's error."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (torch.rand((N, K // g), device="cuda", generator=gen) * 0.02 + 0.001).bfloat16()
    z = torch.randint(0, 16, (N, K // g), dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    x = torch.empty(M, K, device="cuda").normal_(generator=gen).bfloat16()
    y = torch.full((M, N), float("nan"), device="cuda")
    ws = torch.zeros(moe.moe_linear_w4_workspace_size(M, K, N), dtype=torch.uint8, device="cuda")
    moe.moe_linear_w4(M, K, N, g, x, q, s, z, y, ws)
    assert moe.moe_read_device_status(ws) == 0 and torch.isfinite(y).all()
    at = torch.cat([torch.arange(40), torch.arange(N // 2, N // 2 + 40), torch.arange(N - 60, N)]).cuda()
    W, xd = unpack_w4(q[at], s[at], None if z is None else z[at]), x.double()
    # a group's sum, then scales and groups: the sums' error is of the size of the products of both
    want, size = xd @ W.t(), (xd.square() @ W.square().t()).sqrt()
    assert ((y[:, at].double() - want).abs() <= tight._c(K) * size + 2.0 ** -24 * want.abs()).all()


def test_quantize_past_32_bits():
    """2.6 G weights: the first, the middle and the last rows' codes and scales, and back."""
    K, N, g = 16384, 160001, 64
    W = torch.empty(K, N, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k in range(0, K, 1024):
        W[k:k + 1024].normal_(0, 0.1, generator=gen)
    q, s = moe.quantize_w4(W, g)
    back = moe.dequantize_w4(q, s)
    for n in (0, 1, N // 2, N - 2, N - 1):
        w = W[:, n].float().view(-1, g)
        scale = (w.abs().amax(1) / 7.0).bfloat16().float()
        codes = ((w / scale[:, None]).round().clamp(-8, 7) + 8).to(torch.uint8).view(-1)
        assert torch.equal(s[n].float(), scale)
        assert torch.equal(q[n], codes[0::2] | (codes[1::2] << 4))
        assert torch.equal(back[:, n], ((codes.float().view(-1, g) - 8) * scale[:, None]).view(-1).bfloat16())
