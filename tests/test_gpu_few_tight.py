"""moe_layer_few's long sums on the GPU against 64 bits, within a bound of the size
of their errors (_few_tight): strips of more stages than the ring holds, of two
lengths, of the shared and the routed experts."""
import pytest
import torch

import mixture_experts_layer_gating_gb300 as moe
from tests import _few_tight as tight
from tests._lib import ensure_library
from tests.test_gpu_few import KINDS, _call, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


def _within(w, T, D, E, k, I, Is, act="swiglu", renorm=True, seed=0):
    cfg = moe.make_config(T, D, E, k, I, Is, act, w_dtype=w, renormalize=renorm)
    d = _inputs(w, T, D, E, k, I, Is, seed=seed)
    ws = moe.alloc_workspace(cfg)
    out = _call(cfg, d, ws)
    again = _call(cfg, d, ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert moe.moe_read_device_status(ws) == 0
    ids = moe.workspace_view(ws, cfg, "topk_ids", (T, k), torch.int32).long()
    logits = moe.workspace_view(ws, cfg, "logits", (T, E), torch.float32)
    assert torch.equal(ids, torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k])
    want, lin, var = tight.layer(d["x"], d["Wg"], None, d["W13"], d["s13"], d["W2"], d["s2"], d["W13s"], d["s13s"],
                                 d["W2s"], d["s2s"], w, k, act, renorm, ids)
    worst, rms = tight.verdict(out, want, lin, var)
    assert worst <= 1 and rms <= 1, f"{worst}, root mean square {rms} of the allowed"


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("T", [2, 12, 32])
def test_layer_long_runs(w, T):
    D, Is = (4096, 2048) if w == "bf16" else (8192, 4096)
    _within(w, T, D, 512, 2, 128, Is, seed=T)
    _within(w, T, 2048, 4, 4, 2048, 0, seed=T)


@pytest.mark.parametrize("w", ["w4_g32", "w4_g64"])
@pytest.mark.parametrize("T,D,E,k,I,Is", [
    (19, 4096, 64, 8, 704, 2112),
    (20, 4096, 32, 4, 1536, 320),
    (3, 8192, 16, 2, 2048, 64),
    (32, 6144, 48, 3, 256, 704),
    (1, 8192, 8, 8, 576, 0),
])
def test_layer_strips_of_two_lengths(w, T, D, E, k, I, Is):
    _within(w, T, D, E, k, I, Is, seed=I)


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("T,D,E,k,I,Is,act,renorm", [
    (1, 2048, 128, 8, 768, 0, "swiglu", True),
    (7, 2816, 128, 8, 768, 2176, "geglu_tanh", False),
    (17, 4096, 32, 6, 1024, 1024, "swiglu", True),
    (32, 4096, 4, 2, 1024, 1024, "geglu_tanh", True),
])
def test_layer_sizes_in_use(w, T, D, E, k, I, Is, act, renorm):
    _within(w, T, D, E, k, I, Is, act, renorm, seed=T)
