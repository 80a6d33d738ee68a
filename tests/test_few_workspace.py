"""What moe_layer_few's scratch asks of the other calls' workspaces: nothing."""
import ctypes

import pytest

import mixture_experts_layer_gating_gb300 as moe
from tests._lib import ensure_library

P = 1 << 20  # a fake, aligned device address: validation fails before any use

LAYERS = [
    # D, E, k, I, I_shared, w_dtype
    (2048, 128, 8, 768, 0, "bf16"),
    (256, 8, 2, 128, 0, "bf16"),
    (8192, 256, 8, 2048, 2048, "fp8_e4m3"),
    (8192, 256, 8, 2048, 2048, "fp8_e4m3_nk"),
    (2816, 128, 8, 704, 2112, "bf16"),
]


@pytest.fixture(scope="module")
def lib():
    return ensure_library()


@pytest.mark.parametrize("D,E,k,I,Is,w", LAYERS)
def test_a_larger_batch_s_workspace_serves_few_tokens(lib, D, E, k, I, Is, w):
    """A workspace of moe_layer's for 64 tokens is large enough for 1 to 32 (the
    next check, of the null pointers, is what refuses the calls)."""
    n = moe.moe_workspace_size(moe.make_config(64, D, E, k, I, Is, w_dtype=w))
    for T in (1, 7, 16, 31, 32, 33, 64):
        cfg = ctypes.byref(moe.make_config(T, D, E, k, I, Is, w_dtype=w))
        assert lib.moe_layer(cfg, *[None] * 12, P, n, None) == -1
        assert lib.moe_route(cfg, None, None, None, None, None, None, P, n, None) == -1
        assert lib.moe_permute(cfg, *[None] * 7, P, n, None) == -1
        assert lib.moe_grouped_ffn(cfg, *[None] * 15, P, n, None) == -1
        assert lib.moe_finalize(cfg, *[None] * 5, P, n, None) == -1


@pytest.mark.parametrize("D,E,k,I,Is,w", LAYERS)
def test_only_moe_layer_few_needs_its_scratch(lib, D, E, k, I, Is, w):
    """moe_layer takes a workspace up to its last region's end (s, 4 T D bytes, and
    for e4m3 weights the regions after it) and refuses one that ends in it;
    moe_layer_few takes the whole size and nothing less."""
    cfg = moe.make_config(16, D, E, k, I, Is, w_dtype=w)
    n = moe.moe_workspace_size(cfg)
    at = moe.moe_workspace_offset(cfg, moe.WS_SLOTS.index("s"))
    assert lib.moe_layer(ctypes.byref(cfg), *[None] * 12, P, at + 4 * 16 * D - 1, None) == -5
    few = lib.moe_layer_few(ctypes.byref(cfg), *[None] * 12, P, n - 1, None)
    assert few == -5
    assert lib.moe_layer_few(ctypes.byref(cfg), *[None] * 12, P, n, None) == -1
    fp8 = w != "bf16"
    end = at + 4 * 16 * D
    if fp8:  # x16, h16, hs16 and their scales, with the shared expert's rows among the experts'
        end += 16 * (2 * D + 4 + (k + 1) * (4 + 2 * I + 4) + 2 * Is + 4) + 8 * 256
    assert lib.moe_layer(ctypes.byref(cfg), *[None] * 12, P, (end + 255) // 256 * 256, None) == -1
    assert n > end
