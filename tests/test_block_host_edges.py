"""Host-side checks of moe_lora's workspace and of the Python wrappers of the
operators around the experts."""
import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests._lib import ensure_library
from tests.test_block_host import INVALID, WORKSPACE, _lora


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
