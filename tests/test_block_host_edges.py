"""Host-side checks of moe_lora's workspace and of the Python wrappers of the
operators around the experts."""
import ctypes

import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests._lib import ensure_library
from tests.test_block_host import INVALID, P, WORKSPACE, _lora


@pytest.fixture(scope="module")
def lib():
    return ensure_library()


# ------------------------------------------------------------------- lora
# (K, N, r, n): the switch to the many-row kernels at 1024 rows, at 64 an adapter, at 2048 and at
# 32 an adapter; one to eight slices of K, of r one to four
LORA_SIZES = [(8192, 8192, 64, 1), (4096, 4096, 64, 8), (1032, 264, 8, 20), (4096, 1024, 256, 40), (8192, 64, 16, 70), (64, 64, 8, 3),
              (2048, 2048, 24, 4), (16384, 512, 40, 300)]


@pytest.mark.parametrize("K,N,r,n", LORA_SIZES)
def test_lora_workspace_holds_smaller_batches(lib, K, N, r, n):
    """Its size never falls as T grows, and what it gives for T is taken with fewer rows (which
    then fails for the x that is not there, behind the check of the workspace)."""
    few = list(range(0, 1030)) + list(range(1030, 3000, 7)) + [4096, 8192, 9599, 9600, 9601, 20000]
    sizes = [moe.moe_lora_workspace_size(T, K, N, r, n) for T in few]
    assert sizes == sorted(sizes)
    for T in (1, 64, 700, 1024, 2048, 2300, 9600, 20000):
        size = moe.moe_lora_workspace_size(T, K, N, r, n)
        for t in few:
            if 0 < t <= T:
                assert _lora(lib, T=t, K=K, N=N, r=r, n=n, x=None, size=size) == INVALID, (T, t)


@pytest.mark.parametrize("K,N,r,n", LORA_SIZES)
def test_lora_workspace_is_what_some_batch_needs(lib, K, N, r, n):
    for T in (1, 64, 700, 1024, 2300):
        size = moe.moe_lora_workspace_size(T, K, N, r, n)
        assert any(_lora(lib, T=t, K=K, N=N, r=r, n=n, x=None, size=size - 1) == WORKSPACE for t in range(1, T + 1))


# --------------------------------------------------------------- wrappers
def test_wrappers_say_which_tensors_they_take(lib):
    """A tensor that has to be there and is not: the wrapper's own error."""
    T, D, E, k, r, n = 3, 256, 64, 4, 8, 2
    x, W, logits = torch.zeros(T, D).bfloat16(), torch.zeros(D, E).bfloat16(), torch.zeros(T, E)
    ids, w, ws = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), torch.zeros(1 << 20, dtype=torch.uint8)
    cfg, gate = moe.make_config(T, D, E, k, 128), moe.make_gate()

    for a in ((x, None, logits, ids), (x, W, None, ids), (x, W, logits, None), (None, None, None, ids)):
        with pytest.raises(ValueError, match="moe_route_gated takes"):
            moe.moe_route_gated(cfg, gate, a[0], a[1], None, None, a[2], a[3], w, ws)
    for a in ((None, x[0]), (x, None)):
        with pytest.raises(ValueError, match="moe_add_rms_norm takes"):
            moe.moe_add_rms_norm(T, D, a[0], None, a[1], 1e-6, None, x)
    good = [x, torch.zeros(T, dtype=torch.int32), torch.zeros(n, r, D).bfloat16(), torch.zeros(n, E, r).bfloat16(), None, None, logits]
    for i in (0, 1, 2, 3, 6):
        a = list(good)
        a[i] = None
        with pytest.raises(ValueError, match="moe_lora takes"):
            moe.moe_lora(T, D, E, r, n, *a, ws)
    with pytest.raises(ValueError, match="moe_block takes"):
        moe.moe_block(cfg, gate, None, None, x[0], 1e-6, W, None, None, W, None, W, None, None, None, None, None, None, x, x, ws)


# ------------------------------------------------------------------ block
@pytest.mark.parametrize("gate", [False, True])
def test_block_asks_for_the_few_token_scratch_only_where_it_uses_it(lib, gate):
    """A workspace of 64 tokens takes moe_block's batches that run moe_layer's kernels, however
    few the tokens (the next check, of the null pointers, is what refuses these calls)."""
    g = ctypes.byref(moe.make_gate()) if gate else None
    for w, most in (("bf16", 4 if gate else 8), ("fp8_e4m3_nk", 16), ("fp8_e4m3_nk_a8", 0), ("fp8_e4m3", 32), ("w4_g64", 32)):
        n = moe.moe_workspace_size(moe.make_config(64, 2048, 128, 8, 768, w_dtype=w))
        for T in (1, 4, 5, 8, 9, 16, 17, 32, 33, 64):
            cfg = moe.make_config(T, 2048, 128, 8, 768, w_dtype=w)
            own = moe.moe_workspace_size(cfg)
            if w[0] == "w" and T > 32:
                continue  # (not taken)
            small = T <= most and n < own
            assert lib.moe_block(ctypes.byref(cfg), g, *[None] * 3, 0.0, *[None] * 14, P, n, None) == (WORKSPACE if small else INVALID), (w, T)
            assert lib.moe_block(ctypes.byref(cfg), g, *[None] * 3, 0.0, *[None] * 14, P, max(n, own), None) == INVALID
            if T <= most:
                assert lib.moe_block(ctypes.byref(cfg), g, *[None] * 3, 0.0, *[None] * 14, P, own - 1, None) == WORKSPACE
