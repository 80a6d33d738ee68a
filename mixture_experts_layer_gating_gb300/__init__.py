"""GB300 (sm_103a) sparse Mixture-of-Experts FFN layer.

Python binding of the C ABI in ``include/moe.h`` (``libmoe_gb300.so``).  The
functions keep the C names and only marshal arguments: tensors become device
pointers, ``None`` becomes NULL, the stream defaults to torch's current
stream.  Every step of the layer runs in the library's CUDA kernels; there is
no fallback of any kind, and loading fails loudly when the library is absent.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
from typing import Optional

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libmoe_gb300.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG_DIR), "include", "moe.h")

MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_FP8_E4M3_NK, MOE_FP8_E4M3_NK_A8 = 0, 1, 2, 3, 4
MOE_W4_G32, MOE_W4_G64, MOE_W4_G128 = 5, 6, 7
MOE_ACT_SWIGLU, MOE_ACT_GEGLU_TANH = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2_SUM = 0, 1
MOE_OK = 0
MOE_DEV_BAD_EXPERT_ID = 0x1
MOE_DEV_BAD_OFFSETS = 0x2
MOE_DEV_BAD_DEST = 0x4
MOE_DEV_NONFINITE_LOGIT = 0x8
MOE_DEV_WAIT_TIMEOUT = 0x10
WS_SLOTS = ["logits", "topk_ids", "topk_w", "counts", "offsets", "sorted_rows", "dest",
            "x_perm", "h", "y_perm", "h_shared", "s", "x16", "tok_inv", "row_inv"]

_DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8_e4m3": MOE_FP8_E4M3,
           "fp8_e4m3_nk": MOE_FP8_E4M3_NK, "fp8_e4m3_nk_a8": MOE_FP8_E4M3_NK_A8,
           "w4_g32": MOE_W4_G32, "w4_g64": MOE_W4_G64, "w4_g128": MOE_W4_G128}
MOE_FEW_MAX_TOKENS = 32  # most tokens of moe_layer_few, most rows of moe_linear_w4
_ACTS = {"swiglu": MOE_ACT_SWIGLU, "geglu_tanh": MOE_ACT_GEGLU_TANH}
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_GROUP_SCORES = {"max": MOE_GROUP_MAX, "top2_sum": MOE_GROUP_TOP2_SUM}


class MoEConfig(ctypes.Structure):
    """Mirror of moe_config_t."""

    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "D", "E", "k", "I", "I_shared", "act", "act_dtype", "w_dtype", "renormalize")]


class MoEGate(ctypes.Structure):
    """Mirror of moe_gate_t."""

    _fields_ = [(n, ctypes.c_int32) for n in ("score", "n_group", "topk_group", "group_score")] + [
        ("scale", ctypes.c_float)]


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} returned {status}: {text}")
        self.status = status


_lib: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_SIGS = {
    "moe_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(MoEConfig)]),
    "moe_workspace_offset": (ctypes.c_size_t, [ctypes.POINTER(MoEConfig), ctypes.c_int]),
    "moe_route": (ctypes.c_int, [ctypes.POINTER(MoEConfig)] + [_P] * 6 + [_P, ctypes.c_size_t, _P]),
    "moe_permute": (ctypes.c_int, [ctypes.POINTER(MoEConfig)] + [_P] * 7 + [_P, ctypes.c_size_t, _P]),
    "moe_grouped_ffn": (ctypes.c_int, [ctypes.POINTER(MoEConfig)] + [_P] * 15 + [_P, ctypes.c_size_t, _P]),
    "moe_finalize": (ctypes.c_int, [ctypes.POINTER(MoEConfig)] + [_P] * 5 + [_P, ctypes.c_size_t, _P]),
    "moe_layer": (ctypes.c_int, [ctypes.POINTER(MoEConfig)] + [_P] * 12 + [_P, ctypes.c_size_t, _P]),
    "moe_read_device_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_layer_launch_count": (ctypes.c_int, [ctypes.POINTER(MoEConfig)]),
    "moe_set_trace_events": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]),
    "moe_permute_noalloc": (ctypes.c_int, [ctypes.POINTER(MoEConfig)] + [_P] * 7 + [_P]),
    "moe_set_option": (ctypes.c_int, [ctypes.c_int, ctypes.c_int]),
    "moe_pack_weights_nk": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "moe_layer_few": (ctypes.c_int, [ctypes.POINTER(MoEConfig)] + [_P] * 12 + [_P, ctypes.c_size_t, _P]),
    "moe_linear_w4_workspace_size": (ctypes.c_size_t, [ctypes.c_int32] * 3),
    "moe_linear_w4": (ctypes.c_int, [ctypes.c_int32] * 4 + [_P] * 5 +
                      [ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "moe_quantize_w4": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_int32, _P, _P, _P]),
    "moe_dequantize_w4": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int32, _P, _P]),
    "moe_route_gated": (ctypes.c_int, [ctypes.POINTER(MoEConfig), ctypes.POINTER(MoEGate)] + [_P] * 7 +
                        [_P, ctypes.c_size_t, _P]),
    "moe_add_rms_norm": (ctypes.c_int, [ctypes.c_int32] * 3 + [_P] * 3 + [ctypes.c_float] + [_P] * 3 +
                         [ctypes.c_int32, _P, _P]),
    "moe_lora_workspace_size": (ctypes.c_size_t, [ctypes.c_int32] * 5),
    "moe_lora": (ctypes.c_int, [ctypes.c_int32] * 5 + [_P] * 7 + [ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "moe_block": (ctypes.c_int, [ctypes.POINTER(MoEConfig), ctypes.POINTER(MoEGate)] + [_P] * 3 + [ctypes.c_float] +
                  [_P] * 14 + [_P, ctypes.c_size_t, _P]),
    "moe_call": (ctypes.c_int, [ctypes.c_int32, ctypes.c_char_p]),
}
# moe_call's calls and the words of their arguments
_NORM, _ROUTE_GATED, _LORA = 0, 1, 2
_NORM_WORDS, _ROUTE_GATED_WORDS, _LORA_WORDS = (struct.Struct(f).pack for f in ("=6qd6q", "=12q", "=16q"))
MOE_OPT_PAIR_TILES = 1
MOE_OPT_GATHER_A = 2
MOE_OPT_DECODE_KERNEL = 3
MOE_OPT_PDL = 4
MOE_OPT_SHARED_STREAM = 5
MOE_OPT_FUSED_COMBINE = 6
MOE_OPT_TILE_ORDER = 7
MOE_OPT_SHARED_IN_GEMM = 9
MOE_OPT_FUSED_ROUTING = 10
MOE_OPT_B_PREFETCH = 11
MOE_OPT_DYNAMIC_TILES = 12
MOE_OPT_SHARED_CTAS = 13


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmoe_gb300.so (raises when it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with __graft_entry__.build() "
                           "(or python -m mixture_experts_layer_gating_gb300._build)")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = lib
    return lib


def header_symbols(header: str = HEADER_PATH):
    """Function names declared in include/moe.h."""
    txt = open(header).read()
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(moe_\w+)\s*\(", txt, flags=re.M)))


def make_config(T: int, D: int, E: int, k: int, I: int, I_shared: int = 0, act: str = "swiglu",
                act_dtype: str = "bf16", w_dtype: str = "bf16", renormalize: bool = True) -> MoEConfig:
    return MoEConfig(T, D, E, k, I, I_shared, _ACTS[act], _DTYPES[act_dtype], _DTYPES[w_dtype],
                     1 if renormalize else 0)


def config_from_shape(shape, fp8_layout: str = "kn") -> MoEConfig:
    """MoEConfig from a workloads.MoEShape-like object.  For fp8 weights,
    fp8_layout "nk" selects MOE_FP8_E4M3_NK (weights packed by pack_weights_nk)
    and "nk_a8" MOE_FP8_E4M3_NK_A8 (the same weights, W8A8 activations)."""
    if fp8_layout not in ("kn", "nk", "nk_a8"):
        raise ValueError("fp8_layout is 'kn', 'nk' or 'nk_a8'")
    w = shape.w_dtype
    if w == "fp8_e4m3" and fp8_layout == "nk":
        w = "fp8_e4m3_nk"
    if w == "fp8_e4m3" and fp8_layout == "nk_a8":
        w = "fp8_e4m3_nk_a8"
    return make_config(shape.T, shape.D, shape.E, shape.k, shape.I, shape.I_shared, shape.act,
                       shape.act_dtype, w, shape.renormalize)


def make_gate(score: str = "sigmoid", n_group: int = 1, topk_group: int = 1, group_score: str = "top2_sum",
              scale: float = 1.0) -> MoEGate:
    """How moe_route_gated and moe_block choose experts (moe_gate_t)."""
    return MoEGate(_SCORES[score], n_group, topk_group, _GROUP_SCORES[group_score], scale)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


def _first_stream() -> int:
    """Finds torch's way to the current stream, once."""
    global _current_stream
    import torch

    # an integer straight away where this torch has it: building a Stream object
    # takes microseconds
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
    _current_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
    return _current_stream()


_current_stream = _first_stream


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _first_launch(t, stream):
    """Finds torch's way to the current device and its stream, once."""
    global _launch
    import torch

    device_of, raw = torch._C._cuda_getDevice, getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def launch(t, stream):
        device = t.get_device()
        if device < 0 or device != device_of():
            raise ValueError("tensor arguments must live on the current CUDA device")
        return device, raw(device) if stream is None and raw else _stream(stream) or 0

    _launch = launch
    return launch(t, stream)


# (device, stream) of a call on tensor t: the current device, on which the kernels are launched, is t's
_launch = _first_launch


def _address(t, device: int):
    """t's address (None: 0); t is contiguous and lives on that device."""
    if t is None:
        return 0
    if t.get_device() != device:
        raise ValueError("tensor arguments must live on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


def _ws(ws):
    return _ptr(ws), getattr(ws, "nbytes", 0)


def _check(fn: str, st: int):
    if st != MOE_OK:
        raise MoEError(fn, st, load_library().moe_status_string(st).decode())


def moe_workspace_size(cfg: MoEConfig) -> int:
    return int(load_library().moe_workspace_size(ctypes.byref(cfg)))


def moe_workspace_offset(cfg: MoEConfig, which: int) -> int:
    return int(load_library().moe_workspace_offset(ctypes.byref(cfg), which))


def moe_layer_launch_count(cfg: MoEConfig) -> int:
    return int(load_library().moe_layer_launch_count(ctypes.byref(cfg)))


def moe_set_trace_events(events) -> None:
    """Record one of ``events`` (torch.cuda.Event) at every kernel boundary of
    the following moe_layer calls; None switches it off."""
    lib = load_library()
    if not events:
        lib.moe_set_trace_events(None, 0)
        moe_set_trace_events._keep = None
        return
    for e in events:  # force creation of the underlying cudaEvent_t
        if e.cuda_event == 0:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    moe_set_trace_events._keep = arr
    lib.moe_set_trace_events(arr, len(events))


def moe_set_option(option: int, value: int) -> int:
    """Set a kernel-variant option (e.g. MOE_OPT_PAIR_TILES); returns the old value."""
    r = int(load_library().moe_set_option(option, value))
    if r < 0:
        raise MoEError("moe_set_option", r, moe_status_string(r))
    return r


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def moe_route(cfg, x, Wg, logit_bias, logits, topk_ids, topk_w, ws, stream=None):
    wp, wb = _ws(ws)
    _check("moe_route", load_library().moe_route(
        ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(logit_bias), _ptr(logits), _ptr(topk_ids),
        _ptr(topk_w), wp, wb, _stream(stream)))


def moe_permute(cfg, topk_ids, x, counts, offsets, sorted_rows, dest, x_perm, ws, stream=None):
    wp, wb = _ws(ws)
    _check("moe_permute", load_library().moe_permute(
        ctypes.byref(cfg), _ptr(topk_ids), _ptr(x), _ptr(counts), _ptr(offsets), _ptr(sorted_rows),
        _ptr(dest), _ptr(x_perm), wp, wb, _stream(stream)))


def moe_permute_noalloc(cfg, topk_ids, x, counts, offsets, sorted_rows, dest, x_perm, stream=None):
    """moe_permute without a workspace, for callers that cannot allocate device
    memory: its scratch is a fixed array inside the library (see include/moe.h
    for the size limit and the rule that overlapping calls race)."""
    _check("moe_permute_noalloc", load_library().moe_permute_noalloc(
        ctypes.byref(cfg), _ptr(topk_ids), _ptr(x), _ptr(counts), _ptr(offsets), _ptr(sorted_rows),
        _ptr(dest), _ptr(x_perm), _stream(stream)))


def moe_grouped_ffn(cfg, x_perm, offsets, W13, s13, W2, s2, h, y_perm, x=None, W13s=None,
                    s13s=None, W2s=None, s2s=None, h_s=None, s_out=None, ws=None, stream=None):
    wp, wb = _ws(ws)
    _check("moe_grouped_ffn", load_library().moe_grouped_ffn(
        ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(W13), _ptr(s13), _ptr(W2), _ptr(s2),
        _ptr(h), _ptr(y_perm), _ptr(x), _ptr(W13s), _ptr(s13s), _ptr(W2s), _ptr(s2s), _ptr(h_s),
        _ptr(s_out), wp, wb, _stream(stream)))


def moe_finalize(cfg, y_perm, dest, topk_w, s, out, ws, stream=None):
    wp, wb = _ws(ws)
    _check("moe_finalize", load_library().moe_finalize(
        ctypes.byref(cfg), _ptr(y_perm), _ptr(dest), _ptr(topk_w), _ptr(s), _ptr(out), wp, wb,
        _stream(stream)))


def moe_layer(cfg, x, Wg, logit_bias, W13, s13, W2, s2, W13s, s13s, W2s, s2s, out, ws, stream=None):
    wp, wb = _ws(ws)
    _check("moe_layer", load_library().moe_layer(
        ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(logit_bias), _ptr(W13), _ptr(s13), _ptr(W2),
        _ptr(s2), _ptr(W13s), _ptr(s13s), _ptr(W2s), _ptr(s2s), _ptr(out), wp, wb,
        _stream(stream)))


def moe_layer_few(cfg, x, Wg, logit_bias, W13, s13, W2, s2, W13s, s13s, W2s, s2s, out, ws, stream=None):
    """moe_layer for 1 to 32 tokens as one kernel launch; also takes 4-bit
    weights (w_dtype "w4_g32", "w4_g64" or "w4_g128", see quantize_w4)."""
    wp, wb = _ws(ws)
    _check("moe_layer_few", load_library().moe_layer_few(
        ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(logit_bias), _ptr(W13), _ptr(s13), _ptr(W2),
        _ptr(s2), _ptr(W13s), _ptr(s13s), _ptr(W2s), _ptr(s2s), _ptr(out), wp, wb,
        _stream(stream)))


def moe_linear_w4_workspace_size(M: int, K: int, N: int) -> int:
    return int(load_library().moe_linear_w4_workspace_size(M, K, N))


_FLOAT_DTYPES = {}


def _float_dtype(t) -> int:
    """moe_dtype_t of a tensor's dtype (-1: none, which the library refuses)."""
    if not _FLOAT_DTYPES:
        import torch

        _FLOAT_DTYPES.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16})
    return _FLOAT_DTYPES.get(t.dtype, -1)


def moe_linear_w4(M: int, K: int, N: int, group: int, x, Wq, scales, zeros, y, ws, stream=None) -> None:
    """y [M, N] (bf16 or fp32) = x [M, K] times 4-bit weights [N, K/2] with
    scales (and zero points, or None) [N, K/group]."""
    y_dtype, nk = _float_dtype(y), N * K
    try:  # (in one expression: a small product takes little longer than its call)
        fits = (group < 1 or x.nbytes >= 2 * M * K and 2 * Wq.nbytes >= nk and group * scales.nbytes >= 2 * nk
                and y.nbytes >= (4 if y_dtype == MOE_F32 else 2) * M * N
                and _FLOAT_DTYPES.get(x.dtype) == MOE_BF16 == _FLOAT_DTYPES.get(scales.dtype)
                and (zeros is None or group * zeros.nbytes >= nk and zeros.itemsize == 1))
    except AttributeError:  # addresses, or None, which the library refuses
        fits = True
    if not fits:
        raise ValueError("moe_linear_w4 takes bf16 x [M, K], codes [N, K/2], bf16 scales [N, K/group], zero points "
                         "of one byte and y [M, N]")
    wp, wb = _ws(ws)
    _check("moe_linear_w4", load_library().moe_linear_w4(
        M, K, N, group, _ptr(x), _ptr(Wq), _ptr(scales), _ptr(zeros), _ptr(y), y_dtype, wp, wb,
        _stream(stream)))


def moe_quantize_w4(W, G: int, K: int, N: int, group: int, Wq, scales, stream=None) -> None:
    _check("moe_quantize_w4", load_library().moe_quantize_w4(
        _ptr(W), _float_dtype(W), G, K, N, group, _ptr(Wq), _ptr(scales), _stream(stream)))


def moe_dequantize_w4(Wq, scales, zeros, G: int, K: int, N: int, group: int, W, stream=None) -> None:
    _check("moe_dequantize_w4", load_library().moe_dequantize_w4(
        _ptr(Wq), _ptr(scales), _ptr(zeros), G, K, N, group, _ptr(W), _stream(stream)))


def quantize_w4(W, group: int = 128, stream=None):
    """(codes [.., N, K/2] uint8, scales [.., N, K/group] bf16) of the bf16 or
    fp32 weights W [K, N] or [G, K, N], written by moe_quantize_w4."""
    import torch

    if W.dim() not in (2, 3):
        raise ValueError("quantize_w4 takes [K, N] or [G, K, N] weights")
    if group not in (32, 64, 128) or W.shape[-2] % group:
        raise ValueError("quantize_w4: groups of 32, 64 or 128, K a multiple of the group")
    lead, (K, N) = tuple(W.shape[:-2]), W.shape[-2:]
    q = torch.empty((*lead, N, K // 2), dtype=torch.uint8, device=W.device)
    s = torch.empty((*lead, N, K // group), dtype=torch.bfloat16, device=W.device)
    moe_quantize_w4(W, lead[0] if lead else 1, K, N, group, q, s, stream)
    return q, s


def dequantize_w4(Wq, scales, zeros=None, stream=None):
    """bf16 weights [.., K, N] of the 4-bit ones, written by moe_dequantize_w4."""
    import torch

    if Wq.dim() not in (2, 3) or Wq.dim() != scales.dim() or Wq.shape[:-1] != scales.shape[:-1]:
        raise ValueError("dequantize_w4 takes [N, K/2] or [G, N, K/2] codes and scales [.., N, K/group] of as many rows")
    if Wq.dtype != torch.uint8 or scales.dtype != torch.bfloat16:
        raise ValueError("dequantize_w4 takes uint8 codes and bf16 scales")
    lead, N, K = tuple(Wq.shape[:-2]), Wq.shape[-2], 2 * Wq.shape[-1]
    if not K or K not in [scales.shape[-1] * g for g in (32, 64, 128)]:
        raise ValueError("dequantize_w4: groups of 32, 64 or 128 inputs")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape):
        raise ValueError("dequantize_w4: zero points are uint8, one for each scale")
    if any(t is not None and t.device != Wq.device for t in (scales, zeros)):
        raise ValueError("dequantize_w4: codes, scales and zero points on one device")
    W = torch.empty((*lead, K, N), dtype=torch.bfloat16, device=Wq.device)
    moe_dequantize_w4(Wq, scales, zeros, lead[0] if lead else 1, K, N, K // scales.shape[-1], W, stream)
    return W


def _f32(t, n: int) -> bool:
    """t is None or n fp32 values."""
    return t is None or t.nbytes >= 4 * n and _FLOAT_DTYPES.get(t.dtype) == MOE_F32


def moe_route_gated(cfg, gate, x, Wg, logit_bias, select_bias, logits, topk_ids, topk_w, ws, stream=None):
    """moe_route with softmax or sigmoid scores, a bias for the choice, groups and a factor (make_gate)."""
    T, E, n = cfg.T, cfg.E, cfg.T * cfg.k
    if (logits is None or _float_dtype(logits) != MOE_F32 or logits.nbytes < 4 * T * E or not _f32(topk_w, n)
            or topk_ids is None or topk_ids.nbytes < 4 * n or topk_ids.itemsize != 4 or topk_ids.is_floating_point() or not _f32(logit_bias, E)
            or not _f32(select_bias, E)
            or x is not None and (_float_dtype(x) != cfg.act_dtype or x.numel() < T * cfg.D or Wg is None
                                  or Wg.dtype is not x.dtype or Wg.numel() < cfg.D * E)):
        raise ValueError("moe_route_gated takes fp32 logits [T, E], weights [T, k] and biases [E], int32 ids [T, k], "
                         "and x [T, D] and Wg [D, E] of act_dtype")
    device, s = _launch(logits, stream)
    st = load_library().moe_call(_ROUTE_GATED, _ROUTE_GATED_WORDS(
        ctypes.addressof(cfg), 0 if gate is None else ctypes.addressof(gate), _address(x, device), _address(Wg, device),
        _address(logit_bias, device), _address(select_bias, device), _address(logits, device), _address(topk_ids, device),
        _address(topk_w, device), _address(ws, device), getattr(ws, "nbytes", 0), s))
    if st:
        _check("moe_route_gated", st)


def moe_block(cfg, gate, x, residual, norm_weight, eps, Wg, logit_bias, select_bias, W13, s13, W2, s2, W13s, s13s,
              W2s, s2s, sum_out, y, out, ws, stream=None):
    """moe_add_rms_norm (norm_weight None: no norm), then moe_layer with the gate's choice (None: softmax top-k)."""
    dt, n = getattr(x, "dtype", None), cfg.T * cfg.D
    if (x is None or _float_dtype(x) != cfg.act_dtype or any(t is not None and (t.dtype is not dt or t.numel() < m) for t, m in
                                                ((x, n), (residual, n), (sum_out, n), (y, n), (out, n),
                                                 (norm_weight, cfg.D), (Wg, cfg.D * cfg.E)))
            or not _f32(logit_bias, cfg.E) or not _f32(select_bias, cfg.E)):
        raise ValueError("moe_block takes x, residual, sum_out, y and out [T, D], norm_weight [D] and Wg [D, E] of "
                         "act_dtype and fp32 biases [E]")
    device, s = _launch(x, stream)
    a = [_address(t, device) for t in (x, residual, norm_weight, Wg, logit_bias, select_bias, W13, s13, W2, s2, W13s, s13s,
                                       W2s, s2s, sum_out, y, out, ws)]
    _check("moe_block", load_library().moe_block(
        ctypes.byref(cfg), None if gate is None else ctypes.byref(gate), *a[:3], eps, *a[3:], getattr(ws, "nbytes", 0), s))


def moe_add_rms_norm(rows: int, D: int, x, residual, weight, eps: float, sum_out, y, q=None, q_scales=None,
                     q_group: int = 0, stream=None) -> None:
    """sum_out = x + residual and its root-mean-square norm times weight, as y (x's type) and / or as e4m3 rows q
    with a scale per row (q_group 0) or per q_group values; None for what is not there or not wanted."""
    # (a small batch takes little longer than its call: no loops, each attribute looked up once)
    t, dt = (None, -1) if x is None else (x.dtype, _float_dtype(x))
    nb = rows * D * (4 if dt == MOE_F32 else 2)
    if (dt < 0 or x.nbytes < nb or weight is None or weight.dtype is not t or rows > 0 and weight.numel() < D
            or residual is not None and (residual.dtype is not t or residual.nbytes < nb)
            or sum_out is not None and (sum_out.dtype is not t or sum_out.nbytes < nb)
            or y is not None and (y.dtype is not t or y.nbytes < nb)
            or q is not None and (q.itemsize != 1 or q.nbytes < rows * D)
            or q_scales is not None and (_float_dtype(q_scales) != MOE_F32
                                         or q_scales.numel() < rows * (D // q_group if q_group > 0 else 1))):
        raise ValueError("moe_add_rms_norm takes x, residual, sum_out and y [rows, D] and weight [D] of one type (bf16 "
                         "or fp32), one-byte q [rows, D] and fp32 scales [rows, D / q_group]")
    device, s = _launch(x, stream)
    st = load_library().moe_call(_NORM, _NORM_WORDS(
        rows, D, dt, _address(x, device), _address(residual, device), _address(weight, device), eps,
        _address(sum_out, device), _address(y, device), _address(q, device), q_group, _address(q_scales, device), s))
    if st:
        _check("moe_add_rms_norm", st)


def moe_lora_workspace_size(T: int, K: int, N: int, r: int, n: int) -> int:
    return int(load_library().moe_lora_workspace_size(T, K, N, r, n))


def moe_lora(T: int, K: int, N: int, r: int, n: int, x, ids, A, B, scales, base, y, ws, stream=None) -> None:
    """y [T, N] (bf16 or fp32) = base (None: 0; y: in place) + scales[a] x A[a]^T B[a]^T with a = ids[t] of each row
    (outside [0, n): no adapter); x [T, K], A [n, r, K] and B [n, N, r] bf16, scales [n] fp32 or None."""
    there = not (x is None or ids is None or A is None or B is None or y is None)
    t, y_dtype, yt = (x.dtype, _float_dtype(y), y.dtype) if there else (None, -1, None)
    yb = T * N * (4 if y_dtype == MOE_F32 else 2)
    if (not there or _float_dtype(x) != MOE_BF16 or A.dtype is not t or B.dtype is not t or x.nbytes < 2 * T * K
            or A.nbytes < 2 * n * r * K or B.nbytes < 2 * n * N * r or y_dtype < 0 or y.nbytes < yb
            or ids.itemsize != 4 or ids.nbytes < 4 * T or ids.is_floating_point()
            or scales is not None and (_float_dtype(scales) != MOE_F32 or scales.nbytes < 4 * n)
            or base is not None and base is not y and (base.dtype is not yt or base.nbytes < yb)):
        raise ValueError("moe_lora takes bf16 x [T, K], A [n, r, K] and B [n, N, r], int32 ids [T], fp32 scales [n], "
                         "y [T, N] and a base of y's type")
    device, s = _launch(x, stream)
    to = _address(y, device)
    st = load_library().moe_call(_LORA, _LORA_WORDS(
        T, K, N, r, n, _address(x, device), _address(ids, device), _address(A, device), _address(B, device),
        _address(scales, device), to if base is y else _address(base, device), to, y_dtype, _address(ws, device),
        getattr(ws, "nbytes", 0), s))
    if st:
        _check("moe_lora", st)


def moe_pack_weights_nk(W, G: int, K: int, N: int, W_nk, stream=None) -> None:
    _check("moe_pack_weights_nk", load_library().moe_pack_weights_nk(
        _ptr(W), G, K, N, _ptr(W_nk), _stream(stream)))


def pack_weights_nk(W, stream=None):
    """A new [G, N, K] (or [N, K]) copy of the one-byte [G, K, N] (or [K, N])
    weight tensor W, written by moe_pack_weights_nk on W's device."""
    import torch

    if W.element_size() != 1:
        raise ValueError("pack_weights_nk takes one-byte (e4m3) weights")
    if W.dim() not in (2, 3):
        raise ValueError("pack_weights_nk takes [K, N] or [G, K, N] weights")
    Wg = W if W.dim() == 3 else W.unsqueeze(0)
    G, K, N = Wg.shape
    out = torch.empty((G, N, K), dtype=W.dtype, device=W.device)
    moe_pack_weights_nk(Wg, G, K, N, out, stream)
    return out if W.dim() == 3 else out[0]


def moe_read_device_status(ws, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error flags."""
    flags = ctypes.c_int32(0)
    st = load_library().moe_read_device_status(_ptr(ws), _stream(stream), ctypes.byref(flags))
    if st not in (MOE_OK, -4):
        _check("moe_read_device_status", st)
    return int(flags.value)


def alloc_workspace(cfg: MoEConfig, device=None):
    """A zero-filled uint8 torch workspace of moe_workspace_size(cfg) bytes."""
    import torch

    n = moe_workspace_size(cfg)
    if n == 0:
        raise ValueError("invalid MoE configuration")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def workspace_view(ws, cfg: MoEConfig, slot: str, shape, dtype):
    """A typed view of one of moe_layer's intermediates inside the workspace."""
    import torch

    off = moe_workspace_offset(cfg, WS_SLOTS.index(slot))
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    return ws[off:off + nbytes].view(dtype).view(*shape)
