"""Host-side checks of moe_layer_few, moe_linear_w4 and the 4-bit weight
conversions: everything refused here is refused before any CUDA call."""
import ctypes

import pytest

import mixture_experts_layer_gating_gb300 as moe
from tests._lib import ensure_library

P = 1 << 20  # a fake, aligned device address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    return ensure_library()


def _layer(lib, cfg, ptrs, ws=P, n=None):
    return lib.moe_layer_few(ctypes.byref(cfg), *ptrs, ws, moe.moe_workspace_size(cfg) if n is None else n, None)


PLAIN = [P, P, None, P, None, P, None, None, None, None, None, P]
SCALED = [P, P, None, P, P, P, P, None, None, None, None, P]


def test_layer_few_refusals(lib):
    cfg = moe.make_config(4, 256, 8, 2, 128)
    for i in (0, 1, 3, 5, 11):  # x, Wg, W13, W2, out
        for bad in (None, P + 8):
            ptrs = list(PLAIN)
            ptrs[i] = bad
            assert _layer(lib, cfg, ptrs) == -1
    for i in (4, 6):  # scales on bf16 weights, none on scaled ones
        ptrs = list(PLAIN)
        ptrs[i] = P
        assert _layer(lib, cfg, ptrs) == -1
    for w in ("fp8_e4m3", "fp8_e4m3_nk", "w4_g32", "w4_g64", "w4_g128"):
        c = moe.make_config(4, 256, 8, 2, 128, w_dtype=w)
        assert _layer(lib, c, PLAIN) == -1
        assert _layer(lib, c, SCALED[:6] + [None] + SCALED[7:]) == -1
        s = moe.make_config(4, 256, 8, 2, 128, I_shared=128, w_dtype=w)
        assert _layer(lib, s, SCALED) == -1                                 # no shared weights
        assert _layer(lib, s, SCALED[:7] + [P, None, P, P, P]) == -1        # no shared scales
    n = moe.moe_workspace_size(cfg)
    assert _layer(lib, cfg, PLAIN, ws=None) == -5
    assert _layer(lib, cfg, PLAIN, ws=P + 16) == -5
    assert _layer(lib, cfg, PLAIN, n=n - 1) == -5
    assert _layer(lib, moe.make_config(33, 256, 8, 2, 128), PLAIN) == -2    # more than 32 tokens
    assert _layer(lib, moe.make_config(4, 256, 8, 2, 128, w_dtype="fp8_e4m3_nk_a8"), SCALED) == -2
    assert _layer(lib, moe.make_config(4, 256, 8, 2, 128, act_dtype="f32", w_dtype="f32"), PLAIN) == -2
    assert _layer(lib, moe.make_config(4, 256, 8, 9, 128), PLAIN, n=1 << 30) == -1
    assert _layer(lib, moe.make_config(0, 256, 8, 2, 128), PLAIN) == 0      # nothing to do


@pytest.mark.parametrize("w,D,I,Is", [("w4_g32", 272, 128, 0), ("w4_g64", 256, 96, 0), ("w4_g128", 256, 128, 64)])
def test_w4_widths_are_whole_groups(lib, w, D, I, Is):
    assert moe.moe_workspace_size(moe.make_config(4, D, 8, 2, I, Is, w_dtype=w)) == 0


def test_other_calls_refuse_w4_experts(lib):
    cfg = moe.make_config(4, 256, 8, 2, 128, w_dtype="w4_g64")
    n = moe.moe_workspace_size(cfg)
    assert lib.moe_layer(ctypes.byref(cfg), *SCALED, P, n, None) == -2
    assert lib.moe_grouped_ffn(ctypes.byref(cfg), P, P, P, P, P, P, P, P, None, None, None, None, None, None,
                               None, P, n, None) == -2
    assert moe.moe_layer_launch_count(cfg) == 0


def test_workspace_keeps_its_regions(lib):
    """moe_layer_few's scratch comes after the regions that were there."""
    few, many = moe.make_config(32, 256, 8, 2, 128), moe.make_config(33, 256, 8, 2, 128)
    assert moe.moe_workspace_size(few) > moe.moe_workspace_offset(few, 11)
    for T in (1, 8, 32):
        cfg = moe.make_config(T, 256, 8, 2, 128)
        offs = [moe.moe_workspace_offset(cfg, i) for i in range(12)]
        assert offs == sorted(offs) and offs[-1] < moe.moe_workspace_size(cfg)
    assert moe.moe_workspace_size(many) > 0


def _linear(lib, M=1, K=256, N=64, g=64, x=P, q=P, s=P, z=None, y=P, dt=moe.MOE_BF16, ws=P, n=1 << 30):
    return lib.moe_linear_w4(M, K, N, g, x, q, s, z, y, dt, ws, n, None)


def test_linear_refusals(lib):
    assert _linear(lib, M=-1) == -1
    assert _linear(lib, M=33) == -2
    assert _linear(lib, K=0) == -1
    assert _linear(lib, K=96) == -1          # not whole groups
    assert _linear(lib, N=0) == -1
    assert _linear(lib, N=2 ** 31 - 511) == -1
    assert moe.moe_linear_w4_workspace_size(32, 256, 2 ** 31 - 511) == 0
    assert 0 < moe.moe_linear_w4_workspace_size(32, 256, 2 ** 31 - 512) < 1 << 30
    for g in (0, 16, 48, 256, -32):
        assert _linear(lib, g=g) == -1
    for name in "xqsy":
        assert _linear(lib, **{name: None}) == -1
        assert _linear(lib, **{name: P + 4}) == -1
    assert _linear(lib, dt=moe.MOE_FP8_E4M3) == -2
    assert _linear(lib, dt=-1) == -2
    assert _linear(lib, ws=None) == -5
    assert _linear(lib, ws=P + 128) == -5
    assert _linear(lib, n=moe.moe_linear_w4_workspace_size(1, 256, 64) - 1) == -5
    assert _linear(lib, M=0) == 0
    for bad in ((33, 256, 64), (1, 100, 64), (1, 256, 0), (-1, 256, 64)):
        assert moe.moe_linear_w4_workspace_size(*bad) == 0


def test_conversion_refusals(lib):
    Q, B = lib.moe_quantize_w4, lib.moe_dequantize_w4
    for G, K, N, g in ((0, 64, 8, 64), (65536, 64, 8, 64), (1, 96, 8, 64), (1, 64, 0, 64), (1, 64, 8, 48)):
        assert Q(P, moe.MOE_BF16, G, K, N, g, P, P, None) == -1
        assert B(P, P, None, G, K, N, g, P, None) == -1
    assert Q(P, moe.MOE_FP8_E4M3, 1, 64, 8, 64, P, P, None) == -2
    for i in range(3):
        ptrs = [P, P, P]
        for bad in (None, P + 8):
            ptrs[i] = bad
            assert Q(ptrs[0], moe.MOE_F32, 1, 64, 8, 64, ptrs[1], ptrs[2], None) == -1
            assert B(ptrs[0], ptrs[1], None, 1, 64, 8, 64, ptrs[2], None) == -1


def test_python_wrappers_check_shapes(lib):
    import torch

    with pytest.raises(ValueError):
        moe.quantize_w4(torch.zeros(64))
    with pytest.raises(ValueError):
        moe.quantize_w4(torch.zeros(96, 8), 64)
    with pytest.raises(ValueError):
        moe.quantize_w4(torch.zeros(64, 8), 16)
    with pytest.raises(ValueError):
        moe.dequantize_w4(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(1, 8, 1))
    with pytest.raises(ValueError):
        moe.quantize_w4(torch.zeros(64, 8), 32)  # not on a CUDA device
