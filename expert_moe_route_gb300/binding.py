"""Thin ctypes binding of libmoe.so (include/moe.h), same names as the C ABI.

Only argument marshalling lives here: torch tensors supply device pointers and
the current CUDA stream; every step of the MoE layer runs in the library's
CUDA kernels.  There is no fallback: if the library cannot be built or loaded,
importing this module raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

MOE_OK = 0
MOE_LOGITS_IN = 0x1
MOE_CHECK = 0x2
MOE_WEIGHTS_PREPACKED = 0x4
MOE_SINGLE_CTA_TILES = 0x8
MOE_SHARED_SERIAL = 0x10
MOE_FP8_DISPATCH = 0x20
MOE_FP8_MX = 0x40
MOE_ACCUMULATE = 0x80
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_BAD_ROUTING", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_CUDA"}

# the C ABI's exported symbols (checked against include/moe.h by the tests)
SYMBOLS = ("moe_status_string", "moe_version", "moe_last_cuda_error", "moe_trace_events",
           "moe_kernel_launches", "moe_selftest_wait_timeout",
           "moe_route", "moe_dispatch", "moe_dispatch_noalloc", "moe_dispatch_fp8",
           "moe_dequant_fp8", "moe_quantize_mx", "moe_dispatch_mx", "moe_grouped_ffn_mx",
           "moe_prepack_weights", "moe_grouped_ffn", "moe_grouped_ffn_fp8",
           "moe_combine", "moe_layer_fwd", "moe_layer_bwd",
           "moe_sort_rows_bound", "moe_sort", "moe_permute", "moe_permute_bwd", "moe_unpermute",
           "moe_unpermute_bwd", "moe_embed", "moe_embed_bwd", "moe_grad_norm", "moe_adamw_step",
           "moe_route_scores", "moe_route_scores_bwd", "moe_quantize_fp8",
           "moe_quantize_fp8_tiles", "moe_product_fp8", "moe_product_fp8_dx",
           "moe_product_fp8_dw")

# moe_dtype_t
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

# moe_stage_t
STAGES = ("gate", "topk", "dispatch", "gateup", "down", "combine", "bwd_route", "bwd_dh", "bwd_dx",
          "bwd_wg2", "bwd_wg13", "bwd_dwg", "bwd_dxc", "shared_fwd", "shared_bwd")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, cuda_error: int = 0):
        extra = f" (cudaError {cuda_error})" if cuda_error else ""
        super().__init__(f"{where}: {STATUS.get(status, status)}{extra}")
        self.status = status
        self.cuda_error = cuda_error


_vp = ctypes.c_void_p
_i = ctypes.c_int
_u = ctypes.c_uint
_szp = ctypes.POINTER(ctypes.c_size_t)


class moe_shared_t(ctypes.Structure):
    _fields_ = [("fs", _i), ("W1", _vp), ("W3", _vp), ("W2", _vp), ("dW1", _vp), ("dW3", _vp),
                ("dW2", _vp)]


class moe_mx_weights_t(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("W1q", "W1s", "W3q", "W3s", "W2q", "W2s")]


class moe_layer_t(ctypes.Structure):
    _fields_ = [("T", _i), ("d", _i), ("E", _i), ("R", _i), ("f", _i), ("w_gate", _vp),
                ("bias", _vp), ("W1", _vp), ("W3", _vp), ("W2", _vp),
                ("shared", ctypes.POINTER(moe_shared_t)),
                ("mx", ctypes.POINTER(moe_mx_weights_t))]


class moe_saved_t(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("logits", "topk_idx", "topk_w", "counts", "offsets", "row_slot",
                                   "slot_row", "x_perm", "a", "b", "h", "o", "sa", "sb", "sh")]


class moe_adamw_tensor_t(ctypes.Structure):
    _fields_ = [("p", _vp), ("master", _vp), ("g", _vp), ("m", _vp), ("v", _vp),
                ("m_scale", _vp), ("v_scale", _vp), ("n", ctypes.c_longlong),
                ("weight_decay", ctypes.c_double), ("p_dtype", _i), ("g_dtype", _i),
                ("state_bits", _i)]


class moe_adamw_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_longlong), ("seed", ctypes.c_uint32)]


class moe_router_t(ctypes.Structure):
    _fields_ = [("score", _i), ("groups", _i), ("top_groups", _i), ("group_keys", _i),
                ("renormalise", _i), ("scale", ctypes.c_float)]


def _declare(lib):
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_status_string.argtypes = [_i]
    lib.moe_version.restype = _i
    lib.moe_version.argtypes = []
    lib.moe_trace_events.restype = _i
    lib.moe_trace_events.argtypes = [ctypes.POINTER(_vp)]
    lib.moe_kernel_launches.restype = ctypes.c_ulonglong
    lib.moe_kernel_launches.argtypes = []
    lib.moe_selftest_wait_timeout.restype = _i
    lib.moe_selftest_wait_timeout.argtypes = [_u, _vp, _vp]
    lib.moe_route.restype = _i
    lib.moe_route.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _szp, _u, _vp]
    lib.moe_dispatch.restype = _i
    lib.moe_dispatch.argtypes = [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _u,
                                 _vp]
    lib.moe_dispatch_noalloc.restype = _i
    lib.moe_dispatch_noalloc.argtypes = [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _u,
                                         _vp]
    lib.moe_dispatch_fp8.restype = _i
    lib.moe_dispatch_fp8.argtypes = [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _szp, _u, _vp]
    lib.moe_dequant_fp8.restype = _i
    lib.moe_dequant_fp8.argtypes = [_vp, _vp, _i, _i, _vp, _vp]
    _ll = ctypes.c_longlong
    lib.moe_quantize_mx.restype = _i
    lib.moe_quantize_mx.argtypes = [_vp, _ll, _i, _vp, _vp, _vp]
    lib.moe_dispatch_mx.restype = _i
    lib.moe_dispatch_mx.argtypes = [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _szp, _u, _vp]
    lib.moe_grouped_ffn_mx.restype = _i
    lib.moe_grouped_ffn_mx.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _vp, _vp, _vp, _vp, _vp, _szp, _u, _vp]
    lib.moe_prepack_weights.restype = _i
    lib.moe_prepack_weights.argtypes = [_vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp]
    lib.moe_grouped_ffn.restype = _i
    lib.moe_grouped_ffn.argtypes = [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _szp, _u, _vp]
    lib.moe_grouped_ffn_fp8.restype = _i
    lib.moe_grouped_ffn_fp8.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _vp, _szp, _u, _vp]
    lib.moe_combine.restype = _i
    lib.moe_combine.argtypes = [_vp, _vp, _vp, _i, _i, _i, _vp, _vp]
    lib.moe_layer_fwd.restype = _i
    lib.moe_layer_fwd.argtypes = [ctypes.POINTER(moe_layer_t), _vp, _vp,
                                  ctypes.POINTER(moe_saved_t), _vp, _szp, _u, _vp]
    lib.moe_layer_bwd.restype = _i
    lib.moe_layer_bwd.argtypes = [ctypes.POINTER(moe_layer_t), _vp, ctypes.POINTER(moe_saved_t),
                                  _vp, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _u, _vp]
    lib.moe_sort_rows_bound.restype = _ll
    lib.moe_sort_rows_bound.argtypes = [_i, _i, _i, _i, _i]
    lib.moe_sort.restype = _i
    lib.moe_sort.argtypes = [_vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _szp, _u, _vp]
    lib.moe_permute.restype = _i
    lib.moe_permute.argtypes = [_vp, _ll, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _ll, _vp]
    lib.moe_permute_bwd.restype = _i
    lib.moe_permute_bwd.argtypes = [_vp, _ll, _vp, _vp, _vp, _ll, _i, _i, _i, _i, _i, _vp, _ll,
                                    _vp, _vp]
    lib.moe_unpermute.restype = _i
    lib.moe_unpermute.argtypes = [_vp, _ll, _vp, _vp, _i, _i, _i, _i, _i, _vp, _ll, _vp]
    lib.moe_unpermute_bwd.restype = _i
    lib.moe_unpermute_bwd.argtypes = [_vp, _ll, _vp, _vp, _vp, _vp, _ll, _i, _i, _i, _i, _i, _vp,
                                      _ll, _vp, _vp]
    _f = ctypes.c_float
    lib.moe_embed.restype = _i
    lib.moe_embed.argtypes = [_vp, _i, _ll, _vp, _ll, _i, _i, _i, _f, _vp, _ll, _i, _vp]
    lib.moe_embed_bwd.restype = _i
    lib.moe_embed_bwd.argtypes = [_vp, _ll, _vp, _i, _ll, _i, _i, _i, _f, _vp, _ll, _i, _vp, _szp,
                                  _u, _vp]
    _list = ctypes.POINTER(moe_adamw_tensor_t)
    lib.moe_grad_norm.restype = _i
    lib.moe_grad_norm.argtypes = [_list, _i, ctypes.c_double, _vp, _vp, _szp, _vp]
    lib.moe_adamw_step.restype = _i
    lib.moe_adamw_step.argtypes = [_list, _i, ctypes.POINTER(moe_adamw_t), _vp, _vp]
    _router = ctypes.POINTER(moe_router_t)
    lib.moe_route_scores.restype = _i
    lib.moe_route_scores.argtypes = [_vp, _ll, _i, _vp, _i, _i, _i, _router, _vp, _vp, _vp]
    lib.moe_route_scores_bwd.restype = _i
    lib.moe_route_scores_bwd.argtypes = [_vp, _ll, _i, _vp, _vp, _i, _i, _i, _router, _vp, _ll, _vp]
    lib.moe_quantize_fp8.restype = _i
    lib.moe_quantize_fp8.argtypes = [_vp, _ll, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]
    lib.moe_quantize_fp8_tiles.restype = _i
    lib.moe_quantize_fp8_tiles.argtypes = [_vp, _i, _i, _i, _i, _vp, _vp, _vp]
    lib.moe_product_fp8.restype = _i
    lib.moe_product_fp8.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _ll, _i, _vp,
                                    _szp, _u, _vp]
    lib.moe_product_fp8_dx.restype = _i
    lib.moe_product_fp8_dx.argtypes = lib.moe_product_fp8.argtypes
    lib.moe_product_fp8_dw.restype = _i
    lib.moe_product_fp8_dw.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _vp, _szp,
                                       _u, _vp]


_LIB = None


def lib():
    """The loaded library (built in-tree on first use)."""
    global _LIB
    if _LIB is None:
        path = _build.build()
        handle = ctypes.CDLL(path)
        _declare(handle)
        _LIB = handle
    return _LIB


def library_path() -> str:
    return _build.LIB


# ---------------------------------------------------------------- marshalling
def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


# the current stream's handle without a Stream object around it (2 us a call less)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(st, where):
    if st != MOE_OK:
        raise MoeError(st, where, int(lib().moe_last_cuda_error()) if st == 6 else 0)


def _dt(t, dtype, name):
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


# ---------------------------------------------------------------- entry points
def route_ws_bytes(T, d, E, R) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_route(None, None, None, T, d, E, R, None, None, None, None, ctypes.byref(n),
                           0, None), "moe_route(ws query)")
    return n.value


def moe_route(x, w_gate, bias, logits, topk_idx, topk_w, ws=None, flags=0, stream=None):
    """Router; ``ws`` may be None with MOE_LOGITS_IN (else see route_ws_bytes)."""
    T, E = logits.shape
    R = topk_idx.shape[1]
    d = x.shape[1] if x is not None else 0
    _dt(x, torch.bfloat16, "x"); _dt(w_gate, torch.float32, "w_gate"); _dt(bias, torch.float32, "bias")
    _dt(logits, torch.float32, "logits"); _dt(topk_idx, torch.int32, "topk_idx")
    _dt(topk_w, torch.float32, "topk_w")
    n = ctypes.c_size_t(0 if ws is None else ws.numel())
    st = lib().moe_route(_p(x), _p(w_gate), _p(bias), T, d, E, R, _p(logits), _p(topk_idx),
                         _p(topk_w), _p(ws), ctypes.byref(n), flags, _stream(stream))
    _check(st, "moe_route")


def dispatch_ws_bytes(T, d, E, R) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_dispatch(None, None, T, d, E, R, None, None, None, None, None, None,
                              ctypes.byref(n), 0, None), "moe_dispatch(ws query)")
    return n.value


def moe_dispatch(x, topk_idx, E, counts, offsets, row_slot, slot_row, x_perm, ws, flags=0,
                 stream=None):
    T, R = topk_idx.shape
    d = x.shape[1] if x is not None else (x_perm.shape[1] if x_perm is not None else 8)
    _dt(x, torch.bfloat16, "x"); _dt(x_perm, torch.bfloat16, "x_perm")
    for name, t in (("topk_idx", topk_idx), ("counts", counts), ("offsets", offsets),
                    ("row_slot", row_slot), ("slot_row", slot_row)):
        _dt(t, torch.int32, name)
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_dispatch(_p(x), _p(topk_idx), T, d, E, R, _p(counts), _p(offsets),
                            _p(row_slot), _p(slot_row), _p(x_perm), _p(ws), ctypes.byref(n),
                            flags, _stream(stream))
    _check(st, "moe_dispatch")


def moe_dispatch_noalloc(x, topk_idx, E, counts, offsets, row_slot, slot_row, x_perm, flags=0,
                         stream=None):
    """moe_dispatch with the library's static scratch (no workspace argument)."""
    T, R = topk_idx.shape
    d = x.shape[1] if x is not None else (x_perm.shape[1] if x_perm is not None else 8)
    _dt(x, torch.bfloat16, "x"); _dt(x_perm, torch.bfloat16, "x_perm")
    for name, t in (("topk_idx", topk_idx), ("counts", counts), ("offsets", offsets),
                    ("row_slot", row_slot), ("slot_row", slot_row)):
        _dt(t, torch.int32, name)
    st = lib().moe_dispatch_noalloc(_p(x), _p(topk_idx), T, d, E, R, _p(counts), _p(offsets),
                                    _p(row_slot), _p(slot_row), _p(x_perm), flags,
                                    _stream(stream))
    _check(st, "moe_dispatch_noalloc")


def moe_dispatch_fp8(x, topk_idx, E, counts, offsets, row_slot, slot_row, xq_perm, xscale_perm,
                     ws, flags=0, stream=None):
    """Block-scaled fp8 dispatch: E4M3 codes (uint8 [N,d]) and fp32 scales [N, d/128]."""
    T, R = topk_idx.shape
    d = x.shape[1]
    _dt(x, torch.bfloat16, "x"); _dt(xq_perm, torch.uint8, "xq_perm")
    _dt(xscale_perm, torch.float32, "xscale_perm")
    for name, t in (("topk_idx", topk_idx), ("counts", counts), ("offsets", offsets),
                    ("row_slot", row_slot), ("slot_row", slot_row)):
        _dt(t, torch.int32, name)
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_dispatch_fp8(_p(x), _p(topk_idx), T, d, E, R, _p(counts), _p(offsets),
                                _p(row_slot), _p(slot_row), _p(xq_perm), _p(xscale_perm), _p(ws),
                                ctypes.byref(n), flags, _stream(stream))
    _check(st, "moe_dispatch_fp8")


def moe_dequant_fp8(xq, xscale, out, stream=None):
    N, d = xq.shape
    _dt(xq, torch.uint8, "xq"); _dt(xscale, torch.float32, "xscale"); _dt(out, torch.bfloat16, "out")
    _check(lib().moe_dequant_fp8(_p(xq), _p(xscale), N, d, _p(out), _stream(stream)),
           "moe_dequant_fp8")


def grouped_ffn_ws_bytes(N, d, f, E) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_grouped_ffn(None, None, N, d, f, E, None, None, None, None, None, None, None,
                                 None, None, ctypes.byref(n), 0, None), "moe_grouped_ffn(ws query)")
    return n.value


def moe_grouped_ffn(x_perm, offsets, W1, W3, W2, h, out, ws, a_save=None, b_save=None, flags=0,
                    stream=None, row_scale=None):
    N, d = x_perm.shape
    E, f, _ = W1.shape
    for name, t in (("x_perm", x_perm), ("W1", W1), ("W3", W3), ("W2", W2), ("h", h),
                    ("out", out), ("a_save", a_save), ("b_save", b_save)):
        _dt(t, torch.bfloat16, name)
    _dt(offsets, torch.int32, "offsets")
    _dt(row_scale, torch.float32, "row_scale")
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_grouped_ffn(_p(x_perm), _p(offsets), N, d, f, E, _p(W1), _p(W3), _p(W2),
                               _p(row_scale), _p(a_save), _p(b_save), _p(h), _p(out), _p(ws),
                               ctypes.byref(n), flags, _stream(stream))
    _check(st, "moe_grouped_ffn")


def grouped_ffn_fp8_ws_bytes(N, d, f, E) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_grouped_ffn_fp8(None, None, None, N, d, f, E, None, None, None, None, None,
                                     None, None, None, None, ctypes.byref(n), 0, None),
           "moe_grouped_ffn_fp8(ws query)")
    return n.value


def moe_grouped_ffn_fp8(xq_perm, xscale_perm, offsets, W1, W3, W2, h, out, ws, a_save=None,
                        b_save=None, flags=0, stream=None, row_scale=None):
    """moe_grouped_ffn on block-scaled fp8 rows (uint8 codes [N, d], fp32 scales [N, d/128])."""
    N, d = xq_perm.shape
    E, f, _ = W1.shape
    _dt(xq_perm, torch.uint8, "xq_perm")
    _dt(xscale_perm, torch.float32, "xscale_perm")
    for name, t in (("W1", W1), ("W3", W3), ("W2", W2), ("h", h), ("out", out),
                    ("a_save", a_save), ("b_save", b_save)):
        _dt(t, torch.bfloat16, name)
    _dt(offsets, torch.int32, "offsets")
    _dt(row_scale, torch.float32, "row_scale")
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_grouped_ffn_fp8(_p(xq_perm), _p(xscale_perm), _p(offsets), N, d, f, E, _p(W1),
                                   _p(W3), _p(W2), _p(row_scale), _p(a_save), _p(b_save), _p(h),
                                   _p(out), _p(ws), ctypes.byref(n), flags, _stream(stream))
    _check(st, "moe_grouped_ffn_fp8")


def mx_scale_row_bytes(K: int) -> int:
    """Bytes per row of microscaled fp8 scales: K/32, rounded up to a multiple of 16."""
    return -(-K // 512) * 16


def moe_quantize_mx(W, codes, scales, stream=None):
    """Microscaled fp8 codes (uint8 [rows, K]) and scales (uint8 [rows, sk]) of a bf16
    matrix [..., K] along its last dimension."""
    K = W.shape[-1]
    rows = W.numel() // K
    _dt(W, torch.bfloat16, "W"); _dt(codes, torch.uint8, "codes"); _dt(scales, torch.uint8, "scales")
    _check(lib().moe_quantize_mx(_p(W), rows, K, _p(codes), _p(scales), _stream(stream)),
           "moe_quantize_mx")


def moe_dispatch_mx(x, topk_idx, E, counts, offsets, row_slot, slot_row, xq_perm, xscale_perm, ws,
                    flags=0, stream=None):
    """Dispatch with rows in microscaled fp8: codes uint8 [N, d], scales uint8 [N, sk(d)]."""
    T, R = topk_idx.shape
    d = x.shape[1]
    _dt(x, torch.bfloat16, "x"); _dt(xq_perm, torch.uint8, "xq_perm")
    _dt(xscale_perm, torch.uint8, "xscale_perm")
    for name, t in (("topk_idx", topk_idx), ("counts", counts), ("offsets", offsets),
                    ("row_slot", row_slot), ("slot_row", slot_row)):
        _dt(t, torch.int32, name)
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_dispatch_mx(_p(x), _p(topk_idx), T, d, E, R, _p(counts), _p(offsets),
                               _p(row_slot), _p(slot_row), _p(xq_perm), _p(xscale_perm), _p(ws),
                               ctypes.byref(n), flags, _stream(stream))
    _check(st, "moe_dispatch_mx")


def grouped_ffn_mx_ws_bytes(N, d, f, E) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_grouped_ffn_mx(None, None, None, N, d, f, E, None, None, None, None, None,
                                    None, None, None, None, None, None, ctypes.byref(n), 0, None),
           "moe_grouped_ffn_mx(ws query)")
    return n.value


def moe_grouped_ffn_mx(xq, xs, offsets, W1q, W1s, W3q, W3s, W2q, W2s, out, ws, hq=None, hs=None,
                       row_scale=None, flags=0, stream=None):
    """The grouped SwiGLU FFN on microscaled fp8 operands (see include/moe.h).
    W1q, W3q: uint8 [E, f, d] (scales [E, f, sk(d)]); W2q: uint8 [E, d, f] (scales [E, d, sk(f)])."""
    N, d = xq.shape
    E, f, _ = W1q.shape
    for name, t in (("xq", xq), ("xs", xs), ("W1q", W1q), ("W1s", W1s), ("W3q", W3q),
                    ("W3s", W3s), ("W2q", W2q), ("W2s", W2s), ("hq", hq), ("hs", hs)):
        _dt(t, torch.uint8, name)
    _dt(out, torch.bfloat16, "out")
    _dt(offsets, torch.int32, "offsets")
    _dt(row_scale, torch.float32, "row_scale")
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_grouped_ffn_mx(_p(xq), _p(xs), _p(offsets), N, d, f, E, _p(W1q), _p(W1s),
                                  _p(W3q), _p(W3s), _p(W2q), _p(W2s), _p(row_scale), _p(hq),
                                  _p(hs), _p(out), _p(ws), ctypes.byref(n), flags, _stream(stream))
    _check(st, "moe_grouped_ffn_mx")


def moe_prepack_weights(W1, W3, W2, W1p, W3p, W2p, stream=None):
    """Forward weight tiles (see include/moe.h); returns nothing, fills W1p, W3p, W2p."""
    E, f, d = W1.shape
    for name, t in (("W1", W1), ("W3", W3), ("W2", W2), ("W1p", W1p), ("W3p", W3p), ("W2p", W2p)):
        _dt(t, torch.bfloat16, name)
    _check(lib().moe_prepack_weights(_p(W1), _p(W3), _p(W2), E, d, f, _p(W1p), _p(W3p), _p(W2p),
                                     _stream(stream)), "moe_prepack_weights")


def moe_combine(expert_out, slot_row, topk_w, y, R, stream=None):
    T, d = y.shape
    _dt(expert_out, torch.bfloat16, "expert_out"); _dt(y, torch.bfloat16, "y")
    _dt(slot_row, torch.int32, "slot_row"); _dt(topk_w, torch.float32, "topk_w")
    st = lib().moe_combine(_p(expert_out), _p(slot_row), _p(topk_w), T, d, R, _p(y),
                           _stream(stream))
    _check(st, "moe_combine")


# ---------------------------------------------------------------- around the layer
def _rows(t, name, dtype=None):
    """(pointer, row stride) of a matrix whose rows are contiguous."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    if t.dtype is not dtype and (dtype is not None or t.dtype not in DTYPES):
        raise TypeError(f"{name} must be {dtype or 'bf16, fp16 or fp32'}, got {t.dtype}")
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1]


def _shape(t, shape, name):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def sort_rows_bound(T, R, E, align=1, capacity=0) -> int:
    """Rows that hold every plan of moe_sort for these arguments."""
    n = int(lib().moe_sort_rows_bound(T, R, E, align, capacity))
    if n < 0:
        raise MoeError(2, "moe_sort_rows_bound")
    return n


def sort_ws_bytes(T, E, R) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_sort(None, T, E, R, 1, 0, 0, None, None, None, None, None, ctypes.byref(n), 0,
                          None), "moe_sort(ws query)")
    return n.value


def moe_sort(topk_idx, E, counts, offsets, row_slot, slot_row, ws, align=1, capacity=0, flags=0,
             stream=None):
    """Plan of an expert sort (see include/moe.h); row_slot has at least
    sort_rows_bound(T, R, E, align, capacity) entries."""
    T, R = topk_idx.shape
    i32 = torch.int32
    if not (topk_idx.dtype is i32 and counts.dtype is i32 and offsets.dtype is i32
            and row_slot.dtype is i32 and slot_row.dtype is i32):
        for name, t in (("topk_idx", topk_idx), ("counts", counts), ("offsets", offsets),
                        ("row_slot", row_slot), ("slot_row", slot_row)):
            _dt(t, i32, name)
    _shape(counts, (E,), "counts"); _shape(offsets, (E + 1,), "offsets")
    if slot_row.numel() != T * R:
        raise ValueError(f"slot_row must have {T * R} entries")
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_sort(_p(topk_idx), T, E, R, align, capacity, row_slot.numel(), _p(counts),
                        _p(offsets), _p(row_slot), _p(slot_row), _p(ws), ctypes.byref(n), flags,
                        _stream(stream))
    _check(st, "moe_sort")


def _plan_args(T, N, w, slot_row, row_slot=None):
    _dt(slot_row, torch.int32, "slot_row")
    shape = slot_row.shape
    if len(shape) != 2 or shape[0] != T:
        raise ValueError(f"slot_row must have shape ({T}, R)")
    if w is not None:
        _dt(w, torch.float32, "w")
        _shape(w, shape, "w")
    if row_slot is not None:
        _dt(row_slot, torch.int32, "row_slot")
        _shape(row_slot, (N,), "row_slot")
    return shape[1]


def moe_permute(x, w, row_slot, slot_row, rows, stream=None):
    """rows[slot_row[t, r]] = w[t, r] * x[t] (w None: a copy); rows without a slot are zero."""
    (px, ldx), (pr, ldr) = _rows(x, "x"), _rows(rows, "rows", x.dtype)
    T, d = x.shape
    N = rows.shape[0]
    _shape(rows, (N, d), "rows")
    R = _plan_args(T, N, w, slot_row, row_slot)
    st = lib().moe_permute(px, ldx, _p(w), _p(row_slot), _p(slot_row), T, d, R, N,
                           DTYPES[x.dtype], pr, ldr, _stream(stream))
    _check(st, "moe_permute")


def moe_permute_bwd(drows, slot_row, w, x, dx, dw, stream=None):
    """dx[t] = sum_r w[t, r] drows[slot_row[t, r]], dw[t, r] = <x[t], drows[slot_row[t, r]]>
    (x and dw None: no weight gradient)."""
    (pr, ldr), (pd, ldd) = _rows(drows, "drows"), _rows(dx, "dx", drows.dtype)
    px, ldx = _rows(x, "x", drows.dtype)
    N, d = drows.shape
    T = dx.shape[0]
    _shape(dx, (T, d), "dx"); _shape(x, (T, d), "x")
    R = _plan_args(T, N, w, slot_row)
    _dt(dw, torch.float32, "dw"); _shape(dw, (T, R), "dw")
    st = lib().moe_permute_bwd(pr, ldr, _p(slot_row), _p(w), px, ldx, T, d, R, N,
                               DTYPES[drows.dtype], pd, ldd, _p(dw), _stream(stream))
    _check(st, "moe_permute_bwd")


def moe_unpermute(rows, slot_row, w, y, stream=None):
    """y[t] = sum_r w[t, r] rows[slot_row[t, r]] (w None: weight 1)."""
    (pr, ldr), (py, ldy) = _rows(rows, "rows"), _rows(y, "y", rows.dtype)
    N, d = rows.shape
    T = y.shape[0]
    _shape(y, (T, d), "y")
    R = _plan_args(T, N, w, slot_row)
    st = lib().moe_unpermute(pr, ldr, _p(slot_row), _p(w), T, d, R, N, DTYPES[rows.dtype], py, ldy,
                             _stream(stream))
    _check(st, "moe_unpermute")


def moe_unpermute_bwd(dy, row_slot, slot_row, w, rows, drows, dw, stream=None):
    """drows[slot_row[t, r]] = w[t, r] dy[t] (zero without a slot), dw[t, r] =
    <dy[t], rows[slot_row[t, r]]> (rows and dw None: no weight gradient)."""
    (py, ldy), (pd, ldd) = _rows(dy, "dy"), _rows(drows, "drows", dy.dtype)
    pr, ldr = _rows(rows, "rows", dy.dtype)
    T, d = dy.shape
    N = drows.shape[0]
    _shape(drows, (N, d), "drows"); _shape(rows, (N, d), "rows")
    R = _plan_args(T, N, w, slot_row, row_slot)
    _dt(dw, torch.float32, "dw"); _shape(dw, (T, R), "dw")
    st = lib().moe_unpermute_bwd(py, ldy, _p(row_slot), _p(slot_row), _p(w), pr, ldr, T, d, R, N,
                                 DTYPES[dy.dtype], pd, ldd, _p(dw), _stream(stream))
    _check(st, "moe_unpermute_bwd")


def _ids(ids):
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    return _p(ids), ids.element_size(), ids.numel()


def moe_embed(ids, table, out, scale=1.0, stream=None):
    """out[i] = scale * table[ids[i]]; zeros where ids[i] is outside the table."""
    (pi, ib, n), (pt, ldt), (po, ldo) = _ids(ids), _rows(table, "table"), _rows(out, "out")
    V, d = table.shape
    _shape(out, (n, d), "out")
    st = lib().moe_embed(pi, ib, n, pt, ldt, V, d, DTYPES[table.dtype], scale, po, ldo,
                         DTYPES[out.dtype], _stream(stream))
    _check(st, "moe_embed")


def embed_bwd_ws_bytes(n, V, d) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().moe_embed_bwd(None, d, None, 4, n, V, d, 0, 1.0, None, d, 0, None,
                               ctypes.byref(b), 0, None), "moe_embed_bwd(ws query)")
    return b.value


def moe_embed_bwd(dout, ids, dtable, ws, scale=1.0, accumulate=False, flags=0, stream=None):
    """dtable[v] (+)= scale * sum of the rows of dout whose id is v; negative ids contribute
    nothing."""
    (pi, ib, n), (pd, ldd), (pt, ldt) = _ids(ids), _rows(dout, "dout"), _rows(dtable, "dtable")
    V, d = dtable.shape
    _shape(dout, (n, d), "dout")
    b = ctypes.c_size_t(ws.numel())
    st = lib().moe_embed_bwd(pd, ldd, pi, ib, n, V, d, DTYPES[dout.dtype], scale, pt, ldt,
                             DTYPES[dtable.dtype], _p(ws), ctypes.byref(b),
                             flags | (MOE_ACCUMULATE if accumulate else 0), _stream(stream))
    _check(st, "moe_embed_bwd")


class AdamWTensor:
    """One tensor of an optimiser step (moe_adamw_tensor_t).  fp32 m and v: 32-bit states;
    uint8 or float8_e4m3fn m and v with fp32 scales, one per 256 elements: 8-bit states.
    Zeros are the state before the first step."""

    def __init__(self, p, g, m, v, master=None, m_scale=None, v_scale=None, weight_decay=0.0):
        n = p.numel()
        for name, t in (("g", g), ("m", m), ("v", v), ("master", master)):
            if t is not None and t.numel() != n:
                raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
        for name, t in (("p", p), ("g", g)):
            if t.dtype not in (torch.bfloat16, torch.float32):
                raise TypeError(f"{name} must be bf16 or fp32, got {t.dtype}")
        _dt(master, torch.float32, "master")
        codes = (torch.uint8, torch.float8_e4m3fn)
        if m.dtype != v.dtype or (m.dtype != torch.float32 and m.dtype not in codes):
            raise TypeError(f"m and v must both be fp32 or both 8-bit codes, got {m.dtype}, {v.dtype}")
        bits = 8 if m.dtype in codes else 32
        for name, t in (("m_scale", m_scale), ("v_scale", v_scale)):
            if (t is None) != (bits == 32):
                raise ValueError(f"{name} goes with 8-bit states only")
            if t is not None and (t.dtype != torch.float32 or t.numel() != -(-n // 256)):
                raise ValueError(f"{name} must be fp32 with {-(-n // 256)} elements")
        self.tensors = (p, master, g, m, v, m_scale, v_scale)
        self.c = moe_adamw_tensor_t(_p(p), _p(master), _p(g), _p(m), _p(v), _p(m_scale),
                                    _p(v_scale), n, weight_decay, DTYPES[p.dtype],
                                    DTYPES[g.dtype], bits)


class AdamWList:
    """The tensors of an optimiser step: a host array, kept between steps."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.c = (moe_adamw_tensor_t * max(1, len(self.tensors)))(*[t.c for t in self.tensors])

    def __len__(self):
        return len(self.tensors)


def grad_norm_ws_bytes(tensors: AdamWList) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_grad_norm(tensors.c, len(tensors), 0.0, None, None, ctypes.byref(n), None),
           "moe_grad_norm(ws query)")
    return n.value


def moe_grad_norm(tensors: AdamWList, max_norm, norm, ws, stream=None):
    """norm (fp32 [4]) = L2 norm over all gradients, clip factor, 1 if finite, 0."""
    _dt(norm, torch.float32, "norm"); _shape(norm, (4,), "norm")
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_grad_norm(tensors.c, len(tensors), max_norm, _p(norm), _p(ws), ctypes.byref(n),
                             _stream(stream))
    _check(st, "moe_grad_norm")


def moe_adamw_step(tensors: AdamWList, lr, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0,
                   norm=None, stream=None):
    """One AdamW step in place; norm: the record of moe_grad_norm (clip, skip if not finite).
    lr, step and seed are values of the launch: replaying a captured call repeats its step."""
    _dt(norm, torch.float32, "norm"); _shape(norm, (4,), "norm")
    h = moe_adamw_t(lr, beta1, beta2, eps, step, seed)
    st = lib().moe_adamw_step(tensors.c, len(tensors), ctypes.byref(h), _p(norm), _stream(stream))
    _check(st, "moe_adamw_step")


# ---------------------------------------------------------------- routing by scores
class Router:
    """How scores choose experts (moe_router_t): score "softmax" or "sigmoid"; experts in
    `groups` groups of neighbours, of which the best `top_groups` take part, a group's worth
    being the sum of its `group_keys` (1 or 2) largest keys; weights divided by their sum
    (renormalise) and times scale."""

    SCORES = {"softmax": 0, "sigmoid": 1}

    def __init__(self, score="softmax", groups=1, top_groups=1, group_keys=1, renormalise=True,
                 scale=1.0):
        if score not in self.SCORES:
            raise ValueError(f"score must be one of {tuple(self.SCORES)}, got {score!r}")
        self.c = moe_router_t(self.SCORES[score], groups, top_groups, group_keys,
                              int(bool(renormalise)), scale)


def moe_route_scores(logits, router: Router, topk_idx, topk_w, bias=None, stream=None):
    """The R experts of each token by score (+ bias) and their weights (see include/moe.h);
    a logit of -inf closes an expert, slots without one get -1."""
    pl, ldl = _rows(logits, "logits")
    T, E = logits.shape
    _dt(topk_idx, torch.int32, "topk_idx"); _dt(topk_w, torch.float32, "topk_w")
    _dt(bias, torch.float32, "bias"); _shape(bias, (E,), "bias")
    R = topk_idx.shape[1]
    _shape(topk_idx, (T, R), "topk_idx"); _shape(topk_w, (T, R), "topk_w")
    st = lib().moe_route_scores(pl, ldl, DTYPES[logits.dtype], _p(bias), T, E, R,
                                ctypes.byref(router.c), _p(topk_idx), _p(topk_w), _stream(stream))
    _check(st, "moe_route_scores")


def moe_route_scores_bwd(logits, router: Router, topk_idx, dw, dlogits, stream=None):
    """dlogits (every entry) given dw = dL/dtopk_w and the experts that were chosen."""
    (pl, ldl), (pd, ldd) = _rows(logits, "logits"), _rows(dlogits, "dlogits", logits.dtype)
    T, E = logits.shape
    _shape(dlogits, (T, E), "dlogits")
    _dt(topk_idx, torch.int32, "topk_idx"); _dt(dw, torch.float32, "dw")
    R = topk_idx.shape[1]
    _shape(topk_idx, (T, R), "topk_idx"); _shape(dw, (T, R), "dw")
    st = lib().moe_route_scores_bwd(pl, ldl, DTYPES[logits.dtype], _p(topk_idx), _p(dw), T, E, R,
                                    ctypes.byref(router.c), pd, ldd, _stream(stream))
    _check(st, "moe_route_scores_bwd")


# ---------------------------------------------------------------- products on block-scaled fp8
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _codes(t, shape, name):
    if t is None:
        return None
    if t.dtype not in _CODES:
        raise TypeError(f"{name} must be uint8 or float8_e4m3fn, got {t.dtype}")
    _shape(t, shape, name)
    return _p(t)


def _scales(t, shape, name):
    if t is None:
        return None
    _dt(t, torch.float32, name); _shape(t, shape, name)
    return _p(t)


def fp8_blocks(n: int) -> int:
    """Blocks of 128 that cover n elements: the length of a scales' axis."""
    return -(-n // 128)


def moe_quantize_fp8(x, codes=None, scales=None, col_codes=None, col_scales=None, stream=None):
    """E4M3 codes [N, K] and fp32 scales of a matrix: by row (scales [N, ceil(K/128)]), by column
    (col_scales [ceil(N/128), K]) or both in one pass."""
    px, ldx = _rows(x, "x")
    N, K = x.shape
    b = fp8_blocks
    st = lib().moe_quantize_fp8(px, ldx, DTYPES[x.dtype], N, K, _codes(codes, (N, K), "codes"),
                                _scales(scales, (N, b(K)), "scales"),
                                _codes(col_codes, (N, K), "col_codes"),
                                _scales(col_scales, (b(N), K), "col_scales"), _stream(stream))
    _check(st, "moe_quantize_fp8")


def moe_quantize_fp8_tiles(w, codes, scales, stream=None):
    """E4M3 codes of a stack w [E, n, K] with one fp32 scale per 128 x 128 tile
    (scales [E, ceil(n/128), ceil(K/128)])."""
    if w.dtype not in DTYPES:
        raise TypeError(f"w must be bf16, fp16 or fp32, got {w.dtype}")
    E, n, K = w.shape
    st = lib().moe_quantize_fp8_tiles(_p(w), DTYPES[w.dtype], E, n, K,
                                      _codes(codes, (E, n, K), "codes"),
                                      _scales(scales, (E, fp8_blocks(n), fp8_blocks(K)), "scales"),
                                      _stream(stream))
    _check(st, "moe_quantize_fp8_tiles")


def product_fp8_ws_bytes(N, n, K, E=1) -> int:
    """Workspace of the three products of rows [N, K] or [N, n] and weights [E, n, K]."""
    b = ctypes.c_size_t(0)
    _check(lib().moe_product_fp8(None, None, None, N, n, K, E, None, None, None, n, 0, None,
                                 ctypes.byref(b), 0, None), "moe_product_fp8(ws query)")
    return b.value


def _offsets(offsets, E):
    if offsets is None:
        if E != 1:
            raise ValueError(f"{E} experts need offsets")
        return None
    _dt(offsets, torch.int32, "offsets"); _shape(offsets, (E + 1,), "offsets")
    return _p(offsets)


def _product(f, name, a, sa, wq, wscale, out, ws, offsets, flags, stream, back):
    if wq.dim() == 2:
        wq, wscale = wq[None], wscale[None]
    E, n, K = wq.shape
    N = a.shape[0]
    inner, outer = (n, K) if back else (K, n)
    po, ldo = _rows(out, "dx" if back else "out")
    _shape(out, (N, outer), "dx" if back else "out")
    b = ctypes.c_size_t(ws.numel())
    st = f(_codes(a, (N, inner), "dy" if back else "x"),
           _scales(sa, (N, fp8_blocks(inner)), "dy's scales" if back else "x's scales"),
           _offsets(offsets, E), N, n, K, E, _codes(wq, (E, n, K), "w"),
           _scales(wscale, (E, fp8_blocks(n), fp8_blocks(K)), "w's scales"), po, ldo,
           DTYPES[out.dtype], _p(ws), ctypes.byref(b), flags, _stream(stream))
    _check(st, name)


def moe_product_fp8(x, x_scales, w, w_scales, out, ws, offsets=None, flags=0, stream=None):
    """out[i] = x_i w[e]^T for the rows of each expert; x in the row form, w [E, n, K] (or [n, K])
    in tiles; offsets None: one expert, all rows."""
    _product(lib().moe_product_fp8, "moe_product_fp8", x, x_scales, w, w_scales, out, ws, offsets,
             flags, stream, False)


def moe_product_fp8_dx(dy, dy_scales, w, w_scales, dx, ws, offsets=None, flags=0, stream=None):
    """dx[i] = dy_i w[e]: the product's gradient with respect to its rows."""
    _product(lib().moe_product_fp8_dx, "moe_product_fp8_dx", dy, dy_scales, w, w_scales, dx, ws,
             offsets, flags, stream, True)


def moe_product_fp8_dw(dy, dy_scales, x, x_scales, dw, ws, offsets=None, accumulate=False, flags=0,
                       stream=None):
    """dw[e] (+)= dy^T x over the rows of each expert; dy and x in the column form, offsets in
    multiples of 128; dw [E, n, K] (or [n, K])."""
    if dw.dtype not in DTYPES:
        raise TypeError(f"dw must be bf16, fp16 or fp32, got {dw.dtype}")
    E, n, K = dw.shape if dw.dim() == 3 else (1, *dw.shape)
    N = dy.shape[0]
    b = ctypes.c_size_t(ws.numel())
    st = lib().moe_product_fp8_dw(_codes(dy, (N, n), "dy"),
                                  _scales(dy_scales, (fp8_blocks(N), n), "dy's scales"),
                                  _codes(x, (N, K), "x"),
                                  _scales(x_scales, (fp8_blocks(N), K), "x's scales"),
                                  _offsets(offsets, E), N, n, K, E, _p(dw), DTYPES[dw.dtype],
                                  _p(ws), ctypes.byref(b),
                                  flags | (MOE_ACCUMULATE if accumulate else 0), _stream(stream))
    _check(st, "moe_product_fp8_dw")


# ---------------------------------------------------------------- layer
class Shared:
    """A shared expert (moe_shared_t): bf16 weights W1, W3 [fs, d], W2 [d, fs]
    and, for moe_layer_bwd, fp32 gradient buffers of the same shapes."""

    def __init__(self, W1, W3, W2, dW1=None, dW3=None, dW2=None):
        self.W1, self.W3, self.W2 = W1, W3, W2
        self.dW1, self.dW3, self.dW2 = dW1, dW3, dW2
        self.fs = W1.shape[0]
        self.c = moe_shared_t(self.fs, _p(W1), _p(W3), _p(W2), _p(dW1), _p(dW3), _p(dW2))


class MxWeights:
    """The expert weights in microscaled fp8 (moe_mx_weights_t), quantised on the device
    from bf16 W1, W3 [E, f, d] and W2 [E, d, f] with moe_quantize_mx."""

    def __init__(self, W1, W3, W2, stream=None):
        def q(W):
            K = W.shape[-1]
            codes = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
            scales = torch.empty(W.shape[:-1] + (mx_scale_row_bytes(K),), dtype=torch.uint8,
                                 device=W.device)
            moe_quantize_mx(W, codes, scales, stream)
            return codes, scales
        (self.W1q, self.W1s), (self.W3q, self.W3s), (self.W2q, self.W2s) = q(W1), q(W3), q(W2)
        self.c = moe_mx_weights_t(*[_p(getattr(self, n)) for n, _ in moe_mx_weights_t._fields_])


class Layer:
    """Parameters of one MoE layer (device tensors) and their C struct."""

    def __init__(self, w_gate, bias, W1, W3, W2, R, T, shared: Shared = None,
                 mx: MxWeights = None):
        self.w_gate, self.bias, self.W1, self.W3, self.W2 = w_gate, bias, W1, W3, W2
        self.E, self.f, self.d = W1.shape
        self.R, self.T = R, T
        self.shared = shared
        self.mx = mx
        self.c = moe_layer_t(T, self.d, self.E, R, self.f, _p(w_gate), _p(bias), _p(W1), _p(W3),
                             _p(W2), ctypes.pointer(shared.c) if shared is not None else None,
                             ctypes.pointer(mx.c) if mx is not None else None)

    def with_tokens(self, T):
        return Layer(self.w_gate, self.bias, self.W1, self.W3, self.W2, self.R, T, self.shared,
                     self.mx)


class Saved:
    """Caller-owned forward intermediates (allocated here with torch)."""

    def __init__(self, layer: Layer, device, train=True):
        T, d, E, R, f = layer.T, layer.d, layer.E, layer.R, layer.f
        N = T * R
        z = dict(device=device)
        self.logits = torch.empty((T, E), dtype=torch.float32, **z)
        self.topk_idx = torch.empty((T, R), dtype=torch.int32, **z)
        self.topk_w = torch.empty((T, R), dtype=torch.float32, **z)
        self.counts = torch.empty((E,), dtype=torch.int32, **z)
        self.offsets = torch.empty((E + 1,), dtype=torch.int32, **z)
        self.row_slot = torch.empty((N,), dtype=torch.int32, **z)
        self.slot_row = torch.empty((N,), dtype=torch.int32, **z)
        self.x_perm = torch.empty((N, d), dtype=torch.bfloat16, **z)
        self.a = torch.empty((N, f), dtype=torch.bfloat16, **z) if train else None
        self.b = torch.empty((N, f), dtype=torch.bfloat16, **z) if train else None
        self.h = torch.empty((N, f), dtype=torch.bfloat16, **z)
        self.o = torch.empty((N, d), dtype=torch.bfloat16, **z)
        fs = layer.shared.fs if layer.shared is not None else 0
        for n in ("sa", "sb", "sh"):
            setattr(self, n, torch.empty((T, fs), dtype=torch.bfloat16, **z)
                    if fs and train else None)
        self.c = moe_saved_t(*[_p(getattr(self, n)) for n, _ in moe_saved_t._fields_])


def layer_fwd_ws_bytes(layer: Layer, flags=0) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_layer_fwd(ctypes.byref(layer.c), None, None, None, None, ctypes.byref(n),
                               flags, None), "moe_layer_fwd(ws query)")
    return n.value


def layer_bwd_ws_bytes(layer: Layer) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_layer_bwd(ctypes.byref(layer.c), None, None, None, None, None, None, None,
                               None, None, ctypes.byref(n), 0, None), "moe_layer_bwd(ws query)")
    return n.value


def workspace(nbytes: int, device="cuda"):
    """A device byte buffer for the workspace arguments (torch allocates it)."""
    return torch.empty((max(int(nbytes), 256),), dtype=torch.uint8, device=device)


def moe_layer_fwd(layer: Layer, x, y, saved: Saved, ws, flags=0, stream=None):
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_layer_fwd(ctypes.byref(layer.c), _p(x), _p(y), ctypes.byref(saved.c), _p(ws),
                             ctypes.byref(n), flags, _stream(stream))
    _check(st, "moe_layer_fwd")


def moe_layer_bwd(layer: Layer, x, saved: Saved, dy, dx, dW_gate, dW1, dW3, dW2, ws, flags=0,
                  stream=None):
    n = ctypes.c_size_t(ws.numel())
    st = lib().moe_layer_bwd(ctypes.byref(layer.c), _p(x), ctypes.byref(saved.c), _p(dy), _p(dx),
                             _p(dW_gate), _p(dW1), _p(dW3), _p(dW2), _p(ws), ctypes.byref(n),
                             flags, _stream(stream))
    _check(st, "moe_layer_bwd")


class StageTrace:
    """CUDA events recorded by the library around each layer stage (moe_trace_events).

    ``arm()`` makes the library record into this trace's events until
    ``disarm()``; ``elapsed_ms()`` (after the work completed) gives each
    stage's device time, or None for stages that did not run.
    """

    def __init__(self):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * len(STAGES))]
        self._arr = None

    def arm(self):
        # torch creates an event's CUDA handle at its first record(): record every
        # event once (unused stages then read as ~0) before handing the handles over
        for e in self.events:
            e.record()
        self._arr = (_vp * len(self.events))(*[e.cuda_event for e in self.events])
        _check(lib().moe_trace_events(self._arr), "moe_trace_events")

    @staticmethod
    def disarm():
        _check(lib().moe_trace_events(None), "moe_trace_events")

    def elapsed_ms(self):
        out = {}
        for i, name in enumerate(STAGES):
            out[name] = self.events[2 * i].elapsed_time(self.events[2 * i + 1])
        return out


def kernel_launches() -> int:
    return int(lib().moe_kernel_launches())


def status_string(st: int) -> str:
    return lib().moe_status_string(st).decode()


def loaded_path() -> str:
    return os.path.realpath(_build.LIB)
