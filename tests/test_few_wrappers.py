"""Refusals of the Python helpers of the 4-bit forms: what would be read out of
range, or as another type, is refused before any pointer is taken (the tensors here
are on the CPU, which is the last thing refused)."""
import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests._lib import ensure_library


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


def _w4(*lead, N=8, K=128, g=64):
    return torch.zeros(*lead, N, K // 2, dtype=torch.uint8), torch.zeros(*lead, N, K // g, dtype=torch.bfloat16)


@pytest.mark.parametrize("lead", [(), (3,)])
def test_dequantize_compares_codes_scales_and_zeros(lead):
    q, s = _w4(*lead)
    z = torch.zeros(s.shape, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device"):  # right, but not on a GPU
        moe.dequantize_w4(q, s, z)
    fewer = s[..., :4, :].contiguous()
    for bad in (fewer, s.float(), s[..., :1].expand(*lead, 8, 16).contiguous(), s[..., :0]):
        with pytest.raises(ValueError, match="dequantize_w4"):
            moe.dequantize_w4(q, bad)
    for bad in (z[..., :4, :].contiguous(), z[..., :1].contiguous(), z.int(), s):
        with pytest.raises(ValueError, match="dequantize_w4"):
            moe.dequantize_w4(q, s, bad)
    with pytest.raises(ValueError, match="dequantize_w4"):
        moe.dequantize_w4(q.int(), s)


def test_dequantize_compares_the_leading_size():
    q, _ = _w4(3)
    _, s = _w4(2)
    with pytest.raises(ValueError, match="dequantize_w4"):
        moe.dequantize_w4(q, s)


def test_dequantize_refuses_empty_rows():
    with pytest.raises(ValueError, match="dequantize_w4"):
        moe.dequantize_w4(torch.zeros(8, 0, dtype=torch.uint8), torch.zeros(8, 0, dtype=torch.bfloat16))


def test_linear_compares_its_tensors_with_its_sizes():
    M, K, N, g = 3, 128, 8, 64
    q, s = _w4(N=N, K=K, g=g)
    good = dict(x=torch.zeros(M, K, dtype=torch.bfloat16), Wq=q, scales=s,
                zeros=torch.zeros(s.shape, dtype=torch.uint8), y=torch.zeros(M, N))
    ws = torch.zeros(moe.moe_linear_w4_workspace_size(M, K, N), dtype=torch.uint8)

    def call(**other):
        a = dict(good, **other)
        moe.moe_linear_w4(M, K, N, g, a["x"], a["Wq"], a["scales"], a["zeros"], a["y"], ws)

    for a in ({}, {"zeros": None}, {"y": torch.zeros(M, N, dtype=torch.bfloat16)}, {"x": torch.zeros(M + 1, K).bfloat16()}):
        with pytest.raises(ValueError, match="CUDA device"):
            call(**a)
    for name, t in good.items():
        with pytest.raises(ValueError, match="moe_linear_w4 takes"):
            call(**{name: t[:-1].contiguous()})
    for name in ("x", "scales", "zeros"):  # of other types
        with pytest.raises(ValueError, match="moe_linear_w4 takes"):
            call(**{name: good[name].float()})


def test_linear_of_no_rows_takes_empty_tensors(lib):
    """An empty tensor has no address."""
    P = 1 << 20
    assert lib.moe_linear_w4(0, 128, 8, 64, None, P, P, None, None, moe.MOE_BF16, P, 1 << 30, None) == 0
    assert lib.moe_linear_w4(0, 128, 8, 64, None, P, P, None, None, moe.MOE_BF16, P, 0, None) == -5
    assert lib.moe_linear_w4(0, 100, 8, 64, None, P, P, None, None, moe.MOE_BF16, P, 1 << 30, None) == -1
