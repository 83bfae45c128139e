"""Python binding of libsvdq: the SVDQuant W4A4 linear layer on MI355X (gfx950).

Argument marshalling only: every step of the layer runs in libsvdq (the host
packing step in its C++ code, the activation step and the linear in its HIP
kernels).  There is no fallback: if the library cannot be loaded, or the GPU
is not a gfx950, the calls raise.

Functions mirror the C ABI in include/svdq.h:

    pack_weights(W, act_absmax, rank=32, prec=INT4)            host, numpy in/out
    pack_residual(W, smooth, down, up, prec=INT4)              host, numpy in/out
    quantize_act(X, smooth, down, prec=INT4, ...)              device, torch tensors
    w4a4_linear(xq, xscale, h, wq, wscale, up, bias, ...)      device, torch tensors
    w4a4_linear_few(...), w4a4_linear_gated(...)                device, torch tensors
    w4a4_linear_requant(...)                                    device, torch tensors
    w4a4_linear_qkv_norm_rope(...)                              device, torch tensors
    awq_pack_weights(W)                                         host, numpy in/out
    awq_w4a16_linear(X, wq, wscale, bias, ...)                  device, torch tensors
    residual_norm(r, y, gate, ..., scale, shift, ...)           device, torch tensors
    lora_plan(index, n_adapters)                                device, torch tensors
    lora_linear(X, A, B, scale, plan, base, ...)                device, torch tensors
    Kv4Cache(pages, page_size, heads, dim, prec)                device buffers of a 4-bit cache
    kv4_append(cache, K, V, slots)                              device, torch tensors
    kv4_read(cache, slots)                                      device, torch tensors
    kv4_attention(Q, cache, block_table, q_start, kv_len, ...)  device, torch tensors
    rope_frequencies(sections, theta, layout)                   host, numpy out
    rope_table(pos, freq, axis)                                 device, torch tensors
    qk_norm_rope(Q, K, cos, sin, ...)                           device, torch tensors
    kv4_rope_append(cache, Q, K, V, cos, sin, slots, ...)       device, torch tensors
    kv4_tree_plan(cache, parent, q_start, kv_len, ...)          device, torch tensors
    kv4_tree_attention(Q, cache, block_table, ..., mask, ...)   device, torch tensors
    kv4_keep_path(cache, path, q_start, kv_len, ...)            device, torch tensors

Device tensors: X bf16 [M][K], smooth fp32 [K], down bf16 [32][K],
up bf16 [N][32], bias bf16 [N] or None, xq uint8 [M][K/2],
xscale fp32 [M][K/64] (INT4) or uint8 [M][K/32] (MXFP4), h fp32 [M][32],
Y bf16 [M][N].  Calls are enqueued on the current torch stream (or `stream`).
"""
from __future__ import annotations

import ctypes
import operator
import os
from typing import Optional

import numpy as np

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# SVDQ_LIBRARY names another build of the same library (the sanitizer
# tests load an address/undefined-behaviour-sanitized build this way)
LIB_PATH = os.environ.get("SVDQ_LIBRARY") or os.path.join(PKG_DIR, "libsvdq.so")

INT4 = 0
MXFP4 = 1
EPI_NONE = 0
EPI_GELU_TANH = 1
ACT_SILU = 0
ACT_GELU_TANH = 1
FEW_MAX_ROWS = 256
NORM_NONE = 0
NORM_RMS = 1
NORM_LAYER = 2
ROPE_ADJACENT = 0
ROPE_HALVES = 1
ROPE_AXES_BLOCKS = 0
ROPE_AXES_SECTIONS = 1
ROPE_AXES_INTERLEAVED = 2
RANK = 32

STATUS = {
    0: "SVDQ_OK", -1: "SVDQ_ERR_INVALID_ARG", -2: "SVDQ_ERR_SHAPE", -3: "SVDQ_ERR_MISALIGNED",
    -4: "SVDQ_ERR_UNSUPPORTED", -5: "SVDQ_ERR_UNSUPPORTED_DEVICE", -6: "SVDQ_ERR_NONFINITE",
    -7: "SVDQ_ERR_HIP", -8: "SVDQ_ERR_SCRATCH",
}
EXPORTS = ("svdq_status_string", "svdq_version", "svdq_check_device", "svdq_pack_weights",
           "svdq_pack_residual", "svdq_quantize_act", "svdq_w4a4_linear", "svdq_requant_workspace_bytes",
           "svdq_w4a4_linear_requant", "svdq_w4a4_linear_qkv_norm_rope", "svdq_awq_pack_weights",
           "svdq_awq_w4a16_linear", "svdq_w4a4_linear_splitk_workspace_bytes", "svdq_w4a4_linear_splitk",
           "svdq_nf4_codebook", "svdq_nf4_pack_weights", "svdq_nf4_dequantize", "svdq_nf4_w4a16_linear",
           "svdq_w4a4_linear_splitk_noalloc", "svdq_residual_norm", "svdq_lora_plan_bytes",
           "svdq_lora_workspace_bytes", "svdq_lora_plan", "svdq_lora_linear", "svdq_kv4_append", "svdq_kv4_read",
           "svdq_kv4_attention_workspace_bytes", "svdq_kv4_attention", "svdq_rope_frequencies", "svdq_rope_table",
           "svdq_qk_norm_rope", "svdq_kv4_rope_append", "svdq_kv4_tree_plan", "svdq_kv4_tree_attention",
           "svdq_kv4_keep_path", "svdq_w4a4_linear_few", "svdq_w4a4_linear_gated")


class SvdqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


_lib = None


def lib():
    """Load libsvdq.so (building it in-tree only when it is absent)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            from .build import build
            build()
        L = ctypes.CDLL(LIB_PATH)
        P, I = ctypes.c_void_p, ctypes.c_int
        L.svdq_status_string.restype = ctypes.c_char_p
        L.svdq_status_string.argtypes = [I]
        L.svdq_version.restype = I
        L.svdq_version.argtypes = []
        L.svdq_check_device.restype = I
        L.svdq_check_device.argtypes = []
        L.svdq_pack_weights.restype = I
        L.svdq_pack_weights.argtypes = [P, P, I, I, I, I, P, P, P, P, P]
        L.svdq_pack_residual.restype = I
        L.svdq_pack_residual.argtypes = [P, P, P, P, I, I, I, I, P, P]
        L.svdq_quantize_act.restype = I
        L.svdq_quantize_act.argtypes = [P, I, I, P, P, I, I, P, P, P, P]
        L.svdq_w4a4_linear.restype = I
        L.svdq_w4a4_linear.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P, P]
        L.svdq_w4a4_linear_few.restype = I
        L.svdq_w4a4_linear_few.argtypes = L.svdq_w4a4_linear.argtypes
        L.svdq_w4a4_linear_gated.restype = I
        L.svdq_w4a4_linear_gated.argtypes = L.svdq_w4a4_linear.argtypes
        L.svdq_w4a4_linear_splitk_workspace_bytes.restype = ctypes.c_size_t
        L.svdq_w4a4_linear_splitk_workspace_bytes.argtypes = [I, I, I, I]
        L.svdq_w4a4_linear_splitk.restype = I
        L.svdq_w4a4_linear_splitk.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P, P, ctypes.c_size_t, P]
        L.svdq_w4a4_linear_splitk_noalloc.restype = I
        L.svdq_w4a4_linear_splitk_noalloc.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P, P]
        L.svdq_requant_workspace_bytes.restype = ctypes.c_size_t
        L.svdq_requant_workspace_bytes.argtypes = [I, I, I, I]
        L.svdq_w4a4_linear_requant.restype = I
        L.svdq_w4a4_linear_requant.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, P, P, P,
                                               ctypes.c_size_t, P]
        L.svdq_w4a4_linear_qkv_norm_rope.restype = I
        L.svdq_w4a4_linear_qkv_norm_rope.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P, P, ctypes.c_float, P, P,
                                                     P, P]
        L.svdq_awq_pack_weights.restype = I
        L.svdq_awq_pack_weights.argtypes = [P, I, I, P, P]
        L.svdq_awq_w4a16_linear.restype = I
        L.svdq_awq_w4a16_linear.argtypes = [P, P, P, P, I, I, I, P, P]
        L.svdq_nf4_codebook.restype = I
        L.svdq_nf4_codebook.argtypes = [P]
        L.svdq_nf4_pack_weights.restype = I
        L.svdq_nf4_pack_weights.argtypes = [P, I, I, P, P, P]
        L.svdq_nf4_dequantize.restype = I
        L.svdq_nf4_dequantize.argtypes = [P, P, P, I, I, P, P]
        L.svdq_nf4_w4a16_linear.restype = I
        L.svdq_nf4_w4a16_linear.argtypes = [P, P, P, P, P, I, I, I, P, P]
        F = ctypes.c_float
        L.svdq_residual_norm.restype = I
        L.svdq_residual_norm.argtypes = [P, I, P, I, I, I, P, P, F, I, P, P, P, P, P, I, I, F, P, P, P]
        Z = ctypes.c_size_t
        L.svdq_lora_plan_bytes.restype = Z
        L.svdq_lora_plan_bytes.argtypes = [I, I]
        L.svdq_lora_workspace_bytes.restype = Z
        L.svdq_lora_workspace_bytes.argtypes = [I, I, I, I]
        L.svdq_lora_plan.restype = I
        L.svdq_lora_plan.argtypes = [P, I, I, P, Z, P]
        L.svdq_lora_linear.restype = I
        L.svdq_lora_linear.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P, Z, P]
        L64 = ctypes.c_int64
        L.svdq_kv4_append.restype = I
        L.svdq_kv4_append.argtypes = [P, P, P, L64, L64, P, I, P]
        L.svdq_kv4_read.restype = I
        L.svdq_kv4_read.argtypes = [P, P, I, P, P, P]
        L.svdq_kv4_attention_workspace_bytes.restype = Z
        L.svdq_kv4_attention_workspace_bytes.argtypes = [P, I, I, I, I, I]
        L.svdq_kv4_attention.restype = I
        L.svdq_kv4_attention.argtypes = [P, P, L64, P, I, P, P, I, I, I, I, I, F, I, I, P, P, P, Z, P]
        D64 = ctypes.c_double
        L.svdq_rope_frequencies.restype = I
        L.svdq_rope_frequencies.argtypes = [P, I, D64, I, P, P]
        L.svdq_rope_table.restype = I
        L.svdq_rope_table.argtypes = [P, I, I, P, P, I, P, P, P]
        L.svdq_qk_norm_rope.restype = I
        L.svdq_qk_norm_rope.argtypes = [P, L64, I, P, L64, I, I, I, P, P, D64, P, P, P, I, I, I, P, L64, P, L64, P]
        L.svdq_kv4_rope_append.restype = I
        L.svdq_kv4_rope_append.argtypes = [P, P, L64, I, P, P, L64, L64, P, P, D64, P, P, P, I, I, I, P, I, P, L64, P]
        L.svdq_kv4_tree_plan.restype = I
        L.svdq_kv4_tree_plan.argtypes = [P, P, P, P, I, I, I, I, I, P, I, P, P, P]
        L.svdq_kv4_tree_attention.restype = I
        L.svdq_kv4_tree_attention.argtypes = [P, P, L64, P, I, P, P, P, I, I, I, I, I, I, F, P, P, P, Z, P]
        L.svdq_kv4_keep_path.restype = I
        L.svdq_kv4_keep_path.argtypes = [P, P, I, P, P, P, I, I, I, P, P]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().svdq_status_string(int(status)).decode()


def version() -> int:
    return lib().svdq_version()


def _check(st: int, where: str):
    if st != 0:
        raise SvdqError(st, where)


def check_device() -> None:
    _check(lib().svdq_check_device(), "svdq_check_device")


def group_of(prec: int) -> int:
    return 64 if prec == INT4 else 32


# ------------------------------------------------------------------ host calls

def _np(a, dtype):
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, ctypes.c_void_p(a.ctypes.data)


def pack_weights(W: np.ndarray, act_absmax: np.ndarray, rank: int = RANK, prec: int = INT4) -> dict:
    """Smoothing, top-r SVD and residual packing of one layer (host)."""
    prec = _prec(prec)
    W, pW = _np(W, np.uint16)
    a, pa = _np(act_absmax, np.float32)
    if W.ndim != 2:
        raise ValueError(f"W must have 2 dimensions, got shape {W.shape}")
    N, K = W.shape
    if a.shape != (K,):
        raise ValueError(f"act_absmax has shape {a.shape}, expected {(K,)}")
    g = group_of(prec)
    smooth = np.zeros(K, np.float32)
    down = np.zeros((rank, K), np.uint16)
    up = np.zeros((N, rank), np.uint16)
    wq = np.zeros((N, K // 2), np.uint8)
    wscale = np.zeros((N, max(K // g, 0)), np.float32 if prec == INT4 else np.uint8)
    st = lib().svdq_pack_weights(pW, pa, N, K, rank, prec, smooth.ctypes.data, down.ctypes.data,
                                 up.ctypes.data, wq.ctypes.data, wscale.ctypes.data)
    _check(st, "svdq_pack_weights")
    return dict(smooth=smooth, down=down, up=up, wq=wq, wscale=wscale)


def pack_residual(W, smooth, down, up, prec: int = INT4):
    W, pW = _np(W, np.uint16)
    s, ps = _np(smooth, np.float32)
    d, pd = _np(down, np.uint16)
    u, pu = _np(up, np.uint16)
    prec = _prec(prec)
    if W.ndim != 2 or d.ndim != 2:
        raise ValueError("W and down must have 2 dimensions")
    N, K = W.shape
    r = d.shape[0]
    for arr, want, name in ((s, (K,), "smooth"), (d, (r, K), "down"), (u, (N, r), "up")):
        if arr.shape != want:
            raise ValueError(f"{name} has shape {arr.shape}, expected {want}")
    g = group_of(prec)
    wq = np.zeros((N, K // 2), np.uint8)
    wscale = np.zeros((N, max(K // g, 0)), np.float32 if prec == INT4 else np.uint8)
    st = lib().svdq_pack_residual(pW, ps, pd, pu, N, K, d.shape[0], prec, wq.ctypes.data,
                                  wscale.ctypes.data)
    _check(st, "svdq_pack_residual")
    return wq, wscale


# ---------------------------------------------------------------- device calls

def _torch():
    import torch
    return torch


def _chk(t, dtypes, name, shape=None):
    """Type, dtype, shape (when given) and contiguity of a tensor argument."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptrs(*specs):
    """Pointers of device tensors given as (tensor, dtypes, name[, shape])
    (None for an absent optional tensor).  Every tensor's type, dtype, shape
    and contiguity are checked before any device check, so a wrong shape is
    reported the same way with or without a GPU."""
    for sp in specs:
        if sp is not None:
            _chk(*sp)
    out = []
    for sp in specs:
        if sp is None:
            out.append(None)
            continue
        t, name = sp[0], sp[2]
        if t.device.type != "cuda":
            raise TypeError(f"{name} must be a device tensor")
        out.append(ctypes.c_void_p(t.data_ptr()))
    return out


def _prec(prec: int) -> int:
    if prec not in (INT4, MXFP4):
        raise ValueError(f"prec must be INT4 ({INT4}) or MXFP4 ({MXFP4}), got {prec}")
    return prec


def _scale_dtypes(prec: int):
    """The one scale dtype each precision takes: fp32 (INT4), E8M0 bytes (MXFP4)."""
    torch = _torch()
    return (torch.float32,) if prec == INT4 else (torch.uint8,)


def _ndim(t, n, name):
    if getattr(t, "ndim", None) != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(getattr(t, 'shape', ()))}")


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def quantize_act(X, smooth, down, prec: int = INT4, xq=None, xscale=None, h=None, stream=None):
    """Fused smoothing + 4-bit quantization + down projection (one kernel)."""
    torch = _torch()
    prec = _prec(prec)
    _ndim(X, 2, "X")
    _ndim(down, 2, "down")
    M, K = X.shape
    r = down.shape[0]
    g = group_of(prec)
    dev = X.device
    if xq is None:
        xq = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    if xscale is None:
        xscale = torch.empty((M, K // g), dtype=torch.float32 if prec == INT4 else torch.uint8, device=dev)
    if h is None:
        h = torch.empty((M, r), dtype=torch.float32, device=dev)
    bf = (torch.bfloat16, torch.int16)
    pX, ps, pd, pq, pxs, ph = _ptrs(
        (X, bf, "X"), (smooth, (torch.float32,), "smooth", (K,)), (down, bf, "down", (r, K)),
        (xq, (torch.uint8,), "xq", (M, K // 2)), (xscale, _scale_dtypes(prec), "xscale", (M, K // g)),
        (h, (torch.float32,), "h", (M, r)))
    st = lib().svdq_quantize_act(pX, M, K, ps, pd, r, prec, pq, pxs, ph, _stream(stream))
    _check(st, "svdq_quantize_act")
    return xq, xscale, h


def _linear_specs(xq, xscale, h, wq, wscale, up, bias, prec):
    """Shapes of the product's operands: M, K from xq, N from wq, r from up;
    every other operand must agree with them."""
    torch = _torch()
    prec = _prec(prec)
    for t, name in ((xq, "xq"), (xscale, "xscale"), (h, "h"), (wq, "wq"), (wscale, "wscale"), (up, "up")):
        _ndim(t, 2, name)
    M, K = xq.shape[0], xq.shape[1] * 2
    N, r = wq.shape[0], up.shape[1]
    g = group_of(prec)
    bf = (torch.bfloat16, torch.int16)
    specs = [(xq, (torch.uint8,), "xq"), (xscale, _scale_dtypes(prec), "xscale", (M, K // g)),
             (h, (torch.float32,), "h", (M, r)), (wq, (torch.uint8,), "wq", (N, K // 2)),
             (wscale, _scale_dtypes(prec), "wscale", (N, K // g)), (up, bf, "up", (N, r)),
             None if bias is None else (bias, bf, "bias", (N,))]
    return M, N, K, r, specs


def w4a4_linear(xq, xscale, h, wq, wscale, up, bias, prec: int = INT4, epi: int = EPI_NONE,
                Y=None, stream=None):
    """4-bit product + low-rank up projection + bias (+ GELU) -> bf16 (one kernel)."""
    torch = _torch()
    M, N, K, r, specs = _linear_specs(xq, xscale, h, wq, wscale, up, bias, prec)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    *ptrs, pY = _ptrs(*specs, (Y, (torch.bfloat16, torch.int16), "Y", (M, N)))
    st = lib().svdq_w4a4_linear(*ptrs, M, N, K, r, prec, epi, pY, _stream(stream))
    _check(st, "svdq_w4a4_linear")
    return Y


def linear_splitk_workspace_bytes(M: int, N: int, K: int, prec: int = MXFP4) -> int:
    """Device scratch bytes that w4a4_linear_splitk needs on the current
    device (0 when the shape is not split)."""
    return int(lib().svdq_w4a4_linear_splitk_workspace_bytes(M, N, K, prec))


def w4a4_linear_splitk(xq, xscale, h, wq, wscale, up, bias, prec: int = MXFP4, epi: int = EPI_NONE,
                       Y=None, work=None, stream=None):
    """w4a4_linear with K split across work items when the tiles cannot fill
    the chip (fp32 partial sums in `work`, summed in slice order).  When
    `work` is None this binding allocates it with torch; pass a preallocated
    tensor of linear_splitk_workspace_bytes(...) bytes in a serving loop."""
    torch = _torch()
    M, N, K, r, specs = _linear_specs(xq, xscale, h, wq, wscale, up, bias, prec)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    need = linear_splitk_workspace_bytes(M, N, K, prec)
    if work is None and need > 0:
        work = torch.empty(need // 4, dtype=torch.float32, device=xq.device)
    wspec = None if work is None else (work, (torch.float32, torch.uint8), "work")
    *ptrs, pY, pwork = _ptrs(*specs, (Y, (torch.bfloat16, torch.int16), "Y", (M, N)), wspec)
    nbytes = 0 if work is None else work.numel() * work.element_size()
    st = lib().svdq_w4a4_linear_splitk(*ptrs, M, N, K, r, prec, epi, pY, pwork, nbytes, _stream(stream))
    _check(st, "svdq_w4a4_linear_splitk")
    return Y


NOALLOC_SCRATCH_BYTES = 64 << 20


def w4a4_linear_splitk_noalloc(xq, xscale, h, wq, wscale, up, bias, prec: int = MXFP4, epi: int = EPI_NONE,
                               Y=None, stream=None):
    """w4a4_linear_splitk without a workspace: the slice sums go to the
    library's static per-GPU scratch buffer (NOALLOC_SCRATCH_BYTES), so the
    library allocates nothing.  Calls that overlap in time on one GPU race.
    With Y given, this binding allocates nothing either."""
    torch = _torch()
    M, N, K, r, specs = _linear_specs(xq, xscale, h, wq, wscale, up, bias, prec)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    *ptrs, pY = _ptrs(*specs, (Y, (torch.bfloat16, torch.int16), "Y", (M, N)))
    st = lib().svdq_w4a4_linear_splitk_noalloc(*ptrs, M, N, K, r, prec, epi, pY, _stream(stream))
    _check(st, "svdq_w4a4_linear_splitk_noalloc")
    return Y


def requant_workspace_bytes(M: int, N: int, rank: int = RANK, prec: int = INT4) -> int:
    """Device scratch bytes that w4a4_linear_requant needs."""
    return int(lib().svdq_requant_workspace_bytes(M, N, rank, prec))


def w4a4_linear_requant(xq, xscale, h, wq, wscale, up, bias, smooth2, down2, prec: int = INT4,
                        epi: int = EPI_NONE, out=None, work=None, stream=None):
    """w4a4_linear whose epilogue writes the next layer's activation codes,
    scales and h (smooth2, down2 of that layer) instead of Y.  Returns
    (xq2, xscale2, h2)."""
    torch = _torch()
    M, N, K, r, specs = _linear_specs(xq, xscale, h, wq, wscale, up, bias, prec)
    g = group_of(prec)
    dev = xq.device
    if out is None:
        scales = (torch.empty((M, N // 64), dtype=torch.float32, device=dev) if prec == INT4
                  else torch.empty((M, N // 32), dtype=torch.uint8, device=dev))
        out = (torch.empty((M, N // 2), dtype=torch.uint8, device=dev), scales,
               torch.empty((M, r), dtype=torch.float32, device=dev))
    xq2, xs2, h2 = out
    nbytes = requant_workspace_bytes(M, N, r, prec)
    if work is None:
        work = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=dev)
    bf = (torch.bfloat16, torch.int16)
    ptrs = _ptrs(*specs, (smooth2, (torch.float32,), "smooth2", (N,)), (down2, bf, "down2", (r, N)),
                 (xq2, (torch.uint8,), "xq2", (M, N // 2)), (xs2, _scale_dtypes(prec), "xscale2", (M, N // g)),
                 (h2, (torch.float32,), "h2", (M, r)), (work, (torch.uint8, torch.float32), "work"))
    st = lib().svdq_w4a4_linear_requant(*ptrs[:7], M, N, K, r, prec, epi, *ptrs[7:],
                                        work.numel() * work.element_size(), _stream(stream))
    _check(st, "svdq_w4a4_linear_requant")
    return xq2, xs2, h2


def w4a4_linear_qkv_norm_rope(xq, xscale, h, wq, wscale, up, bias, norm_q, norm_k, eps: float, rope_cos,
                              rope_sin, prec: int = INT4, Y=None, stream=None):
    """w4a4_linear of a fused QKV projection (N = 3 H 128) with the Q/K
    RMS-norm and rotary embedding applied in its epilogue (one kernel)."""
    torch = _torch()
    M, N, K, r, specs = _linear_specs(xq, xscale, h, wq, wscale, up, bias, prec)
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    bf = (torch.bfloat16, torch.int16)
    ptrs = _ptrs(*specs, (norm_q, bf, "norm_q", (128,)), (norm_k, bf, "norm_k", (128,)),
                 (rope_cos, (torch.float32,), "rope_cos", (M, 64)), (rope_sin, (torch.float32,), "rope_sin", (M, 64)),
                 (Y, bf, "Y", (M, N)))
    st = lib().svdq_w4a4_linear_qkv_norm_rope(*ptrs[:7], M, N, K, r, prec, ptrs[7], ptrs[8], float(eps),
                                              *ptrs[9:], _stream(stream))
    _check(st, "svdq_w4a4_linear_qkv_norm_rope")
    return Y


def awq_pack_weights(W: np.ndarray):
    """Weight-only AWQ W4A16 packing (host): bf16 bits [N][K] ->
    (wq uint8 [N][K/2], wscale fp32 [N][K/64])."""
    W, pW = _np(W, np.uint16)
    if W.ndim != 2:
        raise ValueError(f"W must have 2 dimensions, got shape {W.shape}")
    N, K = W.shape
    wq = np.zeros((N, K // 2), np.uint8)
    wscale = np.zeros((N, max(K // 64, 0)), np.float32)
    st = lib().svdq_awq_pack_weights(pW, N, K, wq.ctypes.data, wscale.ctypes.data)
    _check(st, "svdq_awq_pack_weights")
    return wq, wscale


def awq_w4a16_linear(X, wq, wscale, bias=None, Y=None, stream=None):
    """Weight-only 4-bit linear with bf16 activations -> bf16 (one kernel)."""
    torch = _torch()
    for t, name in ((X, "X"), (wq, "wq"), (wscale, "wscale")):
        _ndim(t, 2, name)
    M, K = X.shape
    N = wq.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    bf = (torch.bfloat16, torch.int16)
    pX, pq, ps, pb, pY = _ptrs((X, bf, "X"), (wq, (torch.uint8,), "wq", (N, K // 2)),
                               (wscale, (torch.float32,), "wscale", (N, K // 64)),
                               None if bias is None else (bias, bf, "bias", (N,)), (Y, bf, "Y", (M, N)))
    st = lib().svdq_awq_w4a16_linear(pX, pq, ps, pb, M, N, K, pY, _stream(stream))
    _check(st, "svdq_awq_w4a16_linear")
    return Y


def nf4_codebook() -> np.ndarray:
    """The 16 NF4 levels (fp32, ascending)."""
    c = np.zeros(16, np.float32)
    _check(lib().svdq_nf4_codebook(c.ctypes.data), "svdq_nf4_codebook")
    return c


def nf4_pack_weights(W: np.ndarray):
    """NF4 weight-only packing (host): bf16 bits [N][K] -> (wq uint8 [N][K/2],
    qabs uint8 [N*K/64], chunk_scale fp32 [ceil(N*K/64/256)])."""
    W, pW = _np(W, np.uint16)
    if W.ndim != 2:
        raise ValueError(f"W must have 2 dimensions, got shape {W.shape}")
    N, K = W.shape
    nb = N * (K // 64)
    wq = np.zeros((N, K // 2), np.uint8)
    qabs = np.zeros(max(nb, 1), np.uint8)[:nb]
    chunk = np.zeros(max((nb + 255) // 256, 1), np.float32)[:(nb + 255) // 256]
    st = lib().svdq_nf4_pack_weights(pW, N, K, wq.ctypes.data, qabs.ctypes.data, chunk.ctypes.data)
    _check(st, "svdq_nf4_pack_weights")
    return wq, qabs, chunk


def _nf4_specs(wq, qabs, chunk):
    torch = _torch()
    _ndim(wq, 2, "wq")
    N, K = wq.shape[0], wq.shape[1] * 2
    nb = N * (K // 64)
    return N, K, [(wq, (torch.uint8,), "wq"), (qabs, (torch.uint8,), "qabs", (nb,)),
                  (chunk, (torch.float32,), "chunk_scale", ((nb + 255) // 256,))]


def nf4_dequantize(wq, qabs, chunk, Wd=None, stream=None):
    """The dequantized NF4 weights as a bf16 tensor [N][K] (one kernel)."""
    torch = _torch()
    N, K, specs = _nf4_specs(wq, qabs, chunk)
    if Wd is None:
        Wd = torch.empty((N, K), dtype=torch.bfloat16, device=wq.device)
    pq, pa, pc, pW = _ptrs(*specs, (Wd, (torch.bfloat16, torch.int16), "Wd", (N, K)))
    _check(lib().svdq_nf4_dequantize(pq, pa, pc, N, K, pW, _stream(stream)), "svdq_nf4_dequantize")
    return Wd


def nf4_w4a16_linear(X, wq, qabs, chunk, bias=None, Y=None, stream=None):
    """Weight-only NF4 linear with bf16 activations -> bf16 (one kernel)."""
    torch = _torch()
    N, K, specs = _nf4_specs(wq, qabs, chunk)
    _ndim(X, 2, "X")
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    bf = (torch.bfloat16, torch.int16)
    pX, pq, pa, pc, pb, pY = _ptrs((X, bf, "X", (M, K)), *specs, None if bias is None else (bias, bf, "bias", (N,)),
                                   (Y, bf, "Y", (M, N)))
    st = lib().svdq_nf4_w4a16_linear(pX, pq, pa, pc, pb, M, N, K, pY, _stream(stream))
    _check(st, "svdq_nf4_w4a16_linear")
    return Y


# The calls below run between the linears, often on a few rows, where the host
# decides the time: their checks are short, and the module and functions they
# need are looked up once.

_T = None        # torch, after the first call
_I32 = 0x7FFFFFFF          # the largest size the C interface takes (ctypes passes the low 32 bits of a larger one on)
_ELEMENTS = 1 << 30        # SVDQ_MAX_ELEMENTS
_MISFIT = (AttributeError, TypeError, ValueError, IndexError)     # of an argument that is no tensor of this form


def _tt():
    global _T, _BF, _F32, _F64, _U8, _INT32, _raw_stream, _current_device
    if _T is None:
        _T = _torch()
        _BF, _F32, _F64, _U8, _INT32 = _T.bfloat16, _T.float32, _T.float64, _T.uint8, _T.int32
        _raw_stream = getattr(_T._C, "_cuda_getCurrentRawStream", None)
        _current_device = getattr(_T._C, "_cuda_getDevice", None)
    return _T


# The calls of a decoding step take about 4 us in the library and its launch, and
# the checks one by one (_arg, _launch) as long again.  So they first ask for
# everything at once, with outputs given or new ones like their inputs, on the
# current stream; what that does not let through goes the way of the single checks,
# which take it or say what is wrong.


def _bad(t, dtype, name, shape):
    """Raises what is wrong with a tensor that failed its check."""
    torch = _tt()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, dtype, name, shape=None):
    """A contiguous tensor of this dtype (and shape); type, dtype, shape and
    contiguity are checked before the device (`_launch`)."""
    try:
        if t.dtype is dtype and (shape is None or t.shape == shape) and t.is_contiguous():
            return t
    except AttributeError:
        pass
    _bad(t, dtype, name, shape)


def _rows_arg(t, dtype, name, shape):
    """A 2-D tensor whose rows are contiguous but may be a stride apart (a
    slice of a wider tensor); returns the stride."""
    try:
        if t.dtype is dtype and t.shape == shape:
            ld, one = t.stride()
            if one == 1 or not t.numel():
                return ld
            raise ValueError(f"{name} must have contiguous rows")
    except AttributeError:
        pass
    _bad(t, dtype, name, shape)


def _bad_device(dev, names, tensors):
    """Raises what is wrong with the tensors' devices."""
    torch = _tt()
    for name, t in zip(names, tensors):
        if t is not None and t.device != dev:
            raise (TypeError(f"{name} must be a device tensor") if t.device.type != "cuda" or dev.type != "cuda"
                   else ValueError(f"{name} is on {t.device}, expected {dev}"))
    if dev.type != "cuda":
        raise TypeError("the tensors must be device tensors")
    raise ValueError(f"the tensors are on {dev}, the current device is {torch.cuda.current_device()}")


def _launch(dev, names, tensors, stream):
    """The stream to launch on; checks that every tensor lies on `dev` and that
    `dev` is the current device (the library launches there)."""
    index = dev.index                                   # None on the CPU
    for t in tensors:
        if t is not None and t.get_device() != index:
            _bad_device(dev, names, tensors)
    C = _T._C
    if index is None or C._cuda_getDevice() != index:
        _bad_device(dev, names, tensors)
    if stream is None:
        return C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _empty(shape, dtype, dev, stream, like=None):
    """A new tensor; with `stream` given it belongs to that stream, on which the
    kernel runs (an int is a raw stream of this device).  `like`: a tensor
    of this shape; if its type fits too, 1 us less than from the shape."""
    torch = _tt()
    if stream is None or dev.type != "cuda":
        if like is not None and like.dtype is dtype and like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream), dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def residual_norm(r, y=None, gate=None, alpha: float = 1.0, post: int = NORM_NONE, post_w=None, pre: int = NORM_RMS,
                  pre_w=None, pre_b=None, scale=None, shift=None, mod_index=None, eps: float = 1e-6, r_out=None,
                  x=None, want_x: bool = True, stream=None):
    """r' = r + alpha gate post(y), x = pre(r') (1 + scale) + shift (one
    kernel).  r, y [M][D]; r bf16 or fp32, y bf16 or None (r' = r); gate,
    scale, shift [B][D] slices of one modulation output (same row stride), row
    of token m by mod_index [M] int32, or B equal runs of tokens.  Returns
    (r', x): r' is `r` itself without y, x is None with want_x=False.  r_out
    may be r (in place)."""
    torch = _T or _tt()
    bf, f32 = torch.bfloat16, torch.float32
    _ndim(r, 2, "r")
    stype = r.dtype
    if stype is not bf and stype is not f32:
        raise TypeError(f"r has dtype {stype}, expected {(bf, f32)}")
    shape, dev = r.shape, r.device
    M, D = shape
    _arg(r, stype, "r")
    if r.numel() >= _ELEMENTS:
        raise SvdqError(-2, "svdq_residual_norm")
    pY = pO = pX = pG = pS = pH = pPost = pPre = pBias = pI = None
    if y is not None:
        pY = _arg(y, bf, "y", shape).data_ptr()
        if r_out is not None:
            _arg(r_out, stype, "r_out", shape)
        else:
            r_out = torch.empty_like(r) if stream is None else _empty(shape, stype, dev, stream)
        pO = r_out.data_ptr()
    elif r_out is not None:
        raise ValueError("r_out without y: nothing to update")
    if want_x:
        if x is not None:
            _arg(x, bf, "x", shape)
        else:
            x = _empty(shape, bf, dev, stream, r if y is None else y)
        pX = x.data_ptr()
    elif x is not None:
        raise ValueError("x given with want_x=False")
    if post_w is not None:
        pPost = _arg(post_w, bf, "post_w", (D,)).data_ptr()
    if pre_w is not None:
        pPre = _arg(pre_w, bf, "pre_w", (D,)).data_ptr()
    if pre_b is not None:
        pBias = _arg(pre_b, bf, "pre_b", (D,)).data_ptr()
    B, ld = 0, D
    if gate is not None or scale is not None or shift is not None:
        B, ld = _mod_rows(D, gate, scale, shift)
        pG, pS, pH = _ptr(gate), _ptr(scale), _ptr(shift)
    if mod_index is not None:
        pI = _arg(mod_index, torch.int32, "mod_index", (M,)).data_ptr()
    raw = _launch(dev, ("y", "gate", "scale", "shift", "mod_index", "post_w", "pre_w", "pre_b", "r_out", "x"),
                  (y, gate, scale, shift, mod_index, post_w, pre_w, pre_b, r_out, x), stream)
    st = lib().svdq_residual_norm(r.data_ptr(), 1 if stype is f32 else 0, pY, M, D, post, pPost, pG, alpha, pre, pPre,
                                  pBias, pS, pH, pI, B, ld, eps, pO, pX, raw)
    if st:
        raise SvdqError(st, "svdq_residual_norm")
    return (r if y is None else r_out), x


def _mod_rows(D, gate, scale, shift):
    """Rows and row stride of the modulation vectors given."""
    B, ld, sets = 0, D, 0
    for t, name in ((gate, "gate"), (scale, "scale"), (shift, "shift")):
        if t is None:
            continue
        if not B:
            _ndim(t, 2, name)
            B = t.shape[0]
            if B == 0:
                raise ValueError(f"{name} has no rows")
        stride = _rows_arg(t, _T.bfloat16, name, (B, D))
        if B > 1:
            if sets and stride != ld:
                raise ValueError("gate, scale and shift must have the same row stride")
            ld = stride
        sets += 1
    if B > _I32 or ld > _I32:
        raise SvdqError(-2, "svdq_residual_norm")
    return B, ld


def _few_args(where, xq, xscale, h, wq, wscale, up, bias, prec, halves, Y, stream):
    """Checks the operands of a linear whose weight has `halves` times its output
    channels; returns Y and the library call's arguments up to K."""
    torch = _T or _tt()
    prec = _prec(prec)
    u8, bf, f32 = torch.uint8, torch.bfloat16, torch.float32
    sdt, g = (f32, 64) if prec == INT4 else (u8, 32)
    _ndim(xq, 2, "xq")
    _ndim(wq, 2, "wq")
    _ndim(up, 2, "up")
    M, KB = xq.shape
    N, r = up.shape
    K = 2 * KB
    if xq.numel() >= _ELEMENTS or wq.numel() >= _ELEMENTS or max(M, N, K, r) > _I32:
        raise SvdqError(-2, where)
    _arg(xq, u8, "xq")
    _arg(xscale, sdt, "xscale", (M, K // g))
    _arg(h, f32, "h", (M, r))
    _arg(wq, u8, "wq", (N, KB))
    _arg(wscale, sdt, "wscale", (N, K // g))
    _arg(up, bf, "up")
    if bias is not None:
        _arg(bias, bf, "bias", (N,))
    if N % halves:
        raise ValueError(f"wq has {N} rows, expected a gate and an up projection of the same size")
    C, dev = N // halves, xq.device
    Y = _empty((M, C), bf, dev, stream) if Y is None else _arg(Y, bf, "Y", (M, C))
    raw = _launch(dev, ("xscale", "h", "wq", "wscale", "up", "bias", "Y"), (xscale, h, wq, wscale, up, bias, Y), stream)
    return Y, prec, raw, (xq.data_ptr(), xscale.data_ptr(), h.data_ptr(), wq.data_ptr(), wscale.data_ptr(),
                          up.data_ptr(), _ptr(bias), M, C, K, r)


def _few_call(where, call, xq, xscale, h, wq, wscale, up, bias, prec, halves, last, Y, stream):
    if _T is None:
        _tt()
    raw = None
    try:
        M, KB = xq.shape
        N, r = up.shape
        C, dev = N // halves, xq.get_device()
        sdt, G = (_F32, KB >> 5) if prec == INT4 else (_U8, KB >> 4)
        if Y is None and stream is None and dev >= 0:
            Y = xq.new_empty((M, C), dtype=_BF)
        if (stream is None and dev >= 0 and dev == _current_device() == wq.get_device() == xscale.get_device()
                == wscale.get_device() == h.get_device() == up.get_device() == Y.get_device()
                and xq.dtype is _U8 and wq.dtype is _U8 and xscale.dtype is sdt and wscale.dtype is sdt
                and h.dtype is _F32 and up.dtype is _BF and Y.dtype is _BF and C * halves == N
                and xscale.shape == (M, G) and h.shape == (M, r) and wq.shape == (N, KB) and wscale.shape == (N, G)
                and Y.shape == (M, C) and xq.is_contiguous() and wq.is_contiguous() and xscale.is_contiguous()
                and wscale.is_contiguous() and h.is_contiguous() and up.is_contiguous() and Y.is_contiguous()
                and (bias is None or (bias.dtype is _BF and bias.shape == (N,) and bias.get_device() == dev
                                      and bias.is_contiguous()))
                and M * KB < _ELEMENTS and N * KB < _ELEMENTS and r == RANK and prec in (INT4, MXFP4)):
            raw = _raw_stream(dev)
    except _MISFIT:
        pass
    if raw is None:
        Y, prec, raw, (_, _, _, _, _, _, _, M, C, K, r) = _few_args(where, xq, xscale, h, wq, wscale, up, bias, prec, halves,
                                                                   Y, stream)
        KB = K // 2
    st = call(xq.data_ptr(), xscale.data_ptr(), h.data_ptr(), wq.data_ptr(), wscale.data_ptr(), up.data_ptr(),
              None if bias is None else bias.data_ptr(), M, C, 2 * KB, r, prec, last, Y.data_ptr(), raw)
    if st:
        raise SvdqError(st, where)
    return Y


def w4a4_linear_few(xq, xscale, h, wq, wscale, up, bias, prec: int = INT4, epi: int = EPI_NONE, Y=None, stream=None):
    """w4a4_linear for few rows (single tokens, drafted tokens; at most
    FEW_MAX_ROWS): one pass over the weights per 64 rows (one kernel)."""
    return _few_call("svdq_w4a4_linear_few", (_lib or lib()).svdq_w4a4_linear_few, xq, xscale, h, wq, wscale, up, bias,
                     prec, 1, epi, Y, stream)


def w4a4_linear_gated(xq, xscale, h, wq, wscale, up, bias, prec: int = INT4, act: int = ACT_SILU, Y=None, stream=None):
    """act(gate) * up of a gated MLP (one kernel): wq, wscale, up and bias hold the
    gate projection's rows, then the up projection's.  Any number of rows; Y [M][F]
    bf16."""
    return _few_call("svdq_w4a4_linear_gated", (_lib or lib()).svdq_w4a4_linear_gated, xq, xscale, h, wq, wscale, up,
                     bias, prec, 2, act, Y, stream)


class LoraPlan:
    """Rows of one step grouped by adapter (`lora_plan`); `buffer` holds it on
    the device, M and n_adapters are the sizes it was made for."""
    __slots__ = ("buffer", "M", "n_adapters")

    def __init__(self, buffer, M: int, n_adapters: int):
        self.buffer, self.M, self.n_adapters = buffer, M, n_adapters


def lora_plan(index, n_adapters: int, plan: Optional[LoraPlan] = None, stream=None) -> LoraPlan:
    """Groups the rows by adapter: index [M] int32, a value outside [0,
    n_adapters) means none (one kernel).  `plan` of the same sizes is
    overwritten in place (as a captured graph needs)."""
    torch = _tt()
    _ndim(index, 1, "index")
    _arg(index, torch.int32, "index")
    M = index.shape[0]
    if M > _I32 or not 0 < n_adapters <= _I32:
        raise SvdqError(-2 if M > _I32 else -4, "svdq_lora_plan")
    if plan is None:
        need = lib().svdq_lora_plan_bytes(M, n_adapters)
        plan = LoraPlan(_empty(max(need, 16), torch.uint8, index.device, stream), M, n_adapters)
    elif not isinstance(plan, LoraPlan):
        raise TypeError("plan must be a LoraPlan (lora_plan)")
    elif plan.M != M or plan.n_adapters != n_adapters:
        raise ValueError(f"plan is for {plan.M} rows and {plan.n_adapters} adapters, not {M} and {n_adapters}")
    dev = index.device
    raw = _launch(dev, ("plan",),
                  (plan.buffer,), stream)
    st = lib().svdq_lora_plan(index.data_ptr(), M, n_adapters, plan.buffer.data_ptr(), plan.buffer.numel(), raw)
    if st:
        raise SvdqError(st, "svdq_lora_plan")
    return plan


def lora_workspace_bytes(M: int, K: int, rank: int, n_adapters: int) -> int:
    """Device scratch bytes that lora_linear needs on the current device."""
    return int(lib().svdq_lora_workspace_bytes(M, K, rank, n_adapters))


def lora_workspace(M: int, K: int, rank: int, n_adapters: int, device="cuda"):
    """A workspace for lora_linear calls of these sizes (uint8 tensor)."""
    torch = _tt()
    return torch.empty(max(lora_workspace_bytes(M, K, rank, n_adapters), 16), dtype=torch.uint8, device=device)


def lora_linear(X, A, B, scale, plan: LoraPlan, base, Y=None, work=None, stream=None):
    """Y = base + scale_a (X A_a^T) B_a^T for the adapter a of every row (two
    kernels).  X [M][K], A [n][rank][K], B [n][N][rank], base [M][N] bf16,
    scale [n] fp32; rows without an adapter keep base.  Y may be base (in
    place).  When `work` is None it is allocated with torch."""
    torch = _tt()
    bf = torch.bfloat16
    _ndim(X, 2, "X")
    _ndim(A, 3, "A")
    _ndim(base, 2, "base")
    M, K = X.shape
    n, R, _ = A.shape
    N = base.shape[1]
    _arg(X, bf, "X")
    _arg(A, bf, "A", (n, R, K))
    _arg(B, bf, "B", (n, N, R))
    _arg(scale, torch.float32, "scale", (n,))
    _arg(base, bf, "base", (M, N))
    if X.numel() >= _ELEMENTS or A.numel() >= _ELEMENTS or B.numel() >= _ELEMENTS or base.numel() >= _ELEMENTS:
        raise SvdqError(-2, "svdq_lora_linear")
    if not isinstance(plan, LoraPlan):
        raise TypeError("plan must be a LoraPlan (lora_plan)")
    if plan.M != M or plan.n_adapters != n:
        raise ValueError(f"plan is for {plan.M} rows and {plan.n_adapters} adapters, not {M} and {n}")
    dev = X.device
    Y = _empty((M, N), bf, dev, stream, base) if Y is None else _arg(Y, bf, "Y", (M, N))
    if work is None:
        work = _empty(max(lora_workspace_bytes(M, K, R, n), 16), torch.uint8, dev, stream)
    else:
        _arg(work, torch.uint8, "work")
    raw = _launch(dev, ("A", "B", "scale", "plan", "base", "Y", "work"),
                  (A, B, scale, plan.buffer, base, Y, work), stream)
    st = lib().svdq_lora_linear(X.data_ptr(), A.data_ptr(), B.data_ptr(), scale.data_ptr(), plan.buffer.data_ptr(),
                                base.data_ptr(), M, N, K, R, n, Y.data_ptr(), work.data_ptr(), work.numel(), raw)
    if st:
        raise SvdqError(st, "svdq_lora_linear")
    return Y


class _Kv4Struct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("dim", ctypes.c_int), ("prec", ctypes.c_int)]


class Kv4Cache:
    """Buffers of a paged 4-bit key / value cache (svdq_kv4_cache): `pages`
    pages of `page_size` tokens (16, 32, 64, 128 or 256), `heads` key heads of
    `dim` channels (64 or 128), INT4 or MXFP4.  The buffers start out
    uninitialized; a token's slot is page * page_size + place."""

    def __init__(self, pages: int, page_size: int, heads: int, dim: int, prec: int = INT4, device="cuda"):
        torch = _tt()
        prec = _prec(prec)
        if page_size not in (16, 32, 64, 128, 256):
            raise ValueError(f"page_size must be 16, 32, 64, 128 or 256, got {page_size}")
        if dim not in (64, 128):
            raise ValueError(f"dim must be 64 or 128, got {dim}")
        if pages < 1 or heads < 1:
            raise ValueError("a cache has at least one page and one head")
        if pages * page_size > 0x7FFFFFFF or heads > 65535:
            raise ValueError(f"{pages} pages of {page_size} tokens and {heads} heads are more than a cache takes")
        self.pages, self.page_size, self.heads, self.dim, self.prec = pages, page_size, heads, dim, prec
        g = dim // group_of(prec)
        sdt = torch.float32 if prec == INT4 else torch.uint8
        runs = page_size // 16
        self._k_codes = torch.empty((pages, heads, runs, 4, 16, dim // 8), dtype=torch.uint8, device=device)
        self._v_codes = torch.empty((pages, heads, runs, 4, 16, dim // 32, 4), dtype=torch.uint8, device=device)
        self._k_scales = torch.empty((pages, heads, runs, g, 16), dtype=sdt, device=device)
        self._v_scales = torch.empty((pages, heads, runs, g, 16), dtype=sdt, device=device)
        self.device = self._k_codes.device
        self.index = self._k_codes.get_device()           # -1 on the CPU
        self._struct = _Kv4Struct(self._k_codes.data_ptr(), self._k_scales.data_ptr(), self._v_codes.data_ptr(),
                                  self._v_scales.data_ptr(), pages, page_size, heads, dim, prec)
        self._ref = ctypes.addressof(self._struct)

    def __reduce__(self):
        raise TypeError("a Kv4Cache cannot be copied or pickled; copy its buffers")

    k_codes = property(lambda self: self._k_codes)
    v_codes = property(lambda self: self._v_codes)
    k_scales = property(lambda self: self._k_scales)
    v_scales = property(lambda self: self._v_scales)


def _heads_arg(t, name, heads, dim):
    """[T][heads][dim] bf16 with contiguous rows; returns T and the row stride."""
    torch = _T or _tt()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {torch.bfloat16}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {('T', heads, dim)}")
    ld, sh, sd = t.stride()
    if (sd != 1 or (heads > 1 and sh != dim)) and t.numel():
        raise ValueError(f"{name} must have contiguous rows of heads")
    # the stride of a single row (or of none) does not matter
    T = shape[0]
    return T, ld if T > 1 else heads * dim


def _cache_arg(cache):
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")
    return cache.device


def kv4_append(cache: Kv4Cache, K, V, slots, stream=None) -> None:
    """Quantizes K, V [T][heads][dim] bf16 (rows may be a stride apart, as in a
    QKV product) into their slots [T] int32; a slot outside the cache skips
    its token.  The slots of one call must differ.  One kernel."""
    dev = _cache_arg(cache)
    T, ldk = _heads_arg(K, "K", cache.heads, cache.dim)
    TV, ldv = _heads_arg(V, "V", cache.heads, cache.dim)
    if TV != T:
        raise ValueError(f"V has shape {tuple(V.shape)}, expected {tuple(K.shape)}")
    _arg(slots, _T.int32, "slots", (T,))
    raw = _launch(dev, ("K", "V", "slots"),
                  (K, V, slots), stream)
    st = lib().svdq_kv4_append(cache._ref, K.data_ptr(), V.data_ptr(), ldk, ldv, slots.data_ptr(), T, raw)
    if st:
        raise SvdqError(st, "svdq_kv4_append")


def kv4_read(cache: Kv4Cache, slots, K=None, V=None, stream=None):
    """The values the cache holds for `slots` [T] int32: (K, V) fp32
    [T][heads][dim]; zeros for a slot outside the cache.  One kernel."""
    torch = _tt()
    dev = _cache_arg(cache)
    _ndim(slots, 1, "slots")
    _arg(slots, torch.int32, "slots")
    T = slots.shape[0]
    shape = (T, cache.heads, cache.dim)
    K = _empty(shape, torch.float32, dev, stream) if K is None else _arg(K, torch.float32, "K", shape)
    V = _empty(shape, torch.float32, dev, stream, K) if V is None else _arg(V, torch.float32, "V", shape)
    raw = _launch(dev, ("slots", "K", "V"),
                  (slots, K, V), stream)
    st = lib().svdq_kv4_read(cache._ref, slots.data_ptr(), T, K.data_ptr(), V.data_ptr(), raw)
    if st:
        raise SvdqError(st, "svdq_kv4_read")
    return K, V


def _bound(v):
    """A bound on lengths (int32 on the device): a larger one is as loose as
    the largest; 0, which the library refuses, for a negative one."""
    return v if 0 <= v <= _I32 else (_I32 if v > 0 else 0)


def kv4_attention_workspace_bytes(cache: Kv4Cache, T: int, B: int, heads_q: int, max_q: int, max_kv: int) -> int:
    """Device scratch bytes that kv4_attention needs for these sizes."""
    max_q, max_kv = _bound(max_q), _bound(max_kv)
    return int(lib().svdq_kv4_attention_workspace_bytes(cache._ref, T, B, heads_q, max_q, max_kv))


def kv4_attention_workspace(cache: Kv4Cache, T: int, B: int, heads_q: int, max_q: int, max_kv: int):
    """A workspace for kv4_attention calls of these sizes (uint8 tensor)."""
    torch = _tt()
    need = kv4_attention_workspace_bytes(cache, T, B, heads_q, max_q, max_kv)
    return torch.empty(max(need, 16), dtype=torch.uint8, device=cache.device)


def kv4_attention(Q, cache: Kv4Cache, block_table, q_start, kv_len, max_q: int, max_kv: int, scale=None,
                  causal: bool = True, window: int = 0, out=None, lse=None, work=None, stream=None):
    """Attention of the last rows of B sequences over their cached tokens.  Q
    [T][heads_q][dim] bf16; block_table [B][pages per sequence], q_start [B +
    1] and kv_len [B] int32; max_q and max_kv bound the rows and keys of a
    sequence and choose how the work is split.  scale defaults to dim^-0.5.
    Returns out (bf16, Q's shape; rows of no sequence keep what it holds,
    anything in a new one); lse [T][heads_q] fp32 is written when given.  When `work` is None it is allocated with torch."""
    torch = _tt()
    i32 = torch.int32
    dev = _cache_arg(cache)
    _ndim(Q, 3, "Q")
    H, D = Q.shape[1], cache.dim
    if H == 0 or H % cache.heads:
        raise ValueError(f"Q has {H} heads, the cache {cache.heads}")
    T, ldq = _heads_arg(Q, "Q", H, D)
    _ndim(block_table, 2, "block_table")
    _arg(block_table, i32, "block_table")
    B, width = block_table.shape
    _arg(q_start, i32, "q_start", (B + 1,))
    _arg(kv_len, i32, "kv_len", (B,))
    if B > _I32 or width > _I32:
        raise SvdqError(-2, "svdq_kv4_attention")
    if window < 0:
        raise SvdqError(-1, "svdq_kv4_attention")
    max_q, max_kv = _bound(max_q), _bound(max_kv)
    out = _empty((T, H, D), torch.bfloat16, dev, stream, Q) if out is None else _arg(
        out, torch.bfloat16, "out", (T, H, D))
    if lse is not None:
        _arg(lse, torch.float32, "lse", (T, H))
    if work is None:
        need = kv4_attention_workspace_bytes(cache, T, B, H, max_q, max_kv)
        work = _empty(need, torch.uint8, dev, stream) if need else None
    else:
        _arg(work, torch.uint8, "work")
    raw = _launch(dev, ("Q", "block_table", "q_start", "kv_len", "out", "lse", "work"),
                  (Q, block_table, q_start, kv_len, out, lse, work), stream)
    st = lib().svdq_kv4_attention(cache._ref, Q.data_ptr(), ldq, block_table.data_ptr(), width, q_start.data_ptr(),
                                  kv_len.data_ptr(), B, T, H, max_q, max_kv, D ** -0.5 if scale is None else scale,
                                  1 if causal else 0, min(window, _I32), out.data_ptr(), _ptr(lse), _ptr(work),
                                  0 if work is None else work.numel(), raw)
    if st:
        raise SvdqError(st, "svdq_kv4_attention")
    return out


def kv4_tree_attention(Q, cache: Kv4Cache, block_table, q_start, kv_len, mask, max_q: int, max_kv: int, scale=None,
                       out=None, lse=None, work=None, stream=None):
    """kv4_attention of drafted tokens: row i of a sequence's n sees the keys
    before place kv_len - n, and of the drafted ones those in its mask [T][words]
    int32 (kv4_tree_plan).  Workspace as for kv4_attention."""
    torch = _T or _tt()
    raw = None
    try:
        T, H, D = Q.shape
        ldq, sh, sd = Q.stride()
        B, width = block_table.shape
        words, dev = mask.shape[1], Q.get_device()
        if (stream is None and out is not None and work is not None and dev >= 0
                and dev == _current_device() == cache.index == block_table.get_device() == q_start.get_device()
                == kv_len.get_device() == mask.get_device() == out.get_device() == work.get_device()
                and Q.dtype is _BF and out.dtype is _BF and block_table.dtype is _INT32 and q_start.dtype is _INT32
                and kv_len.dtype is _INT32 and mask.dtype is _INT32 and work.dtype is _U8 and D == cache.dim and sd == 1
                and sh == D and H and H % cache.heads == 0 and q_start.shape == (B + 1,) and kv_len.shape == (B,)
                and mask.shape == (T, words) and out.shape == Q.shape and out.is_contiguous() and mask.is_contiguous()
                and block_table.is_contiguous() and q_start.is_contiguous() and kv_len.is_contiguous()
                and work.is_contiguous() and 0 <= max_q <= _I32 and 0 <= max_kv <= _I32
                and T < _I32 and B < _I32 and width < _I32 and words < _I32 and H < _I32
                and (lse is None or (lse.dtype is _F32 and lse.shape == (T, H) and lse.get_device() == dev
                                     and lse.is_contiguous()))):
            raw = _raw_stream(dev)
            ldq = ldq if T > 1 else H * D
    except _MISFIT:
        pass
    if raw is None:
        i32 = torch.int32
        dev = _cache_arg(cache)
        _ndim(Q, 3, "Q")
        H, D = Q.shape[1], cache.dim
        if H == 0 or H % cache.heads:
            raise ValueError(f"Q has {H} heads, the cache {cache.heads}")
        T, ldq = _heads_arg(Q, "Q", H, D)
        _ndim(block_table, 2, "block_table")
        _arg(block_table, i32, "block_table")
        B, width = block_table.shape
        _arg(q_start, i32, "q_start", (B + 1,))
        _arg(kv_len, i32, "kv_len", (B,))
        _ndim(mask, 2, "mask")
        words = mask.shape[1]
        _arg(mask, i32, "mask", (T, words))
        if T > _I32 or B > _I32 or H > _I32 or width > _I32 or words > _I32:
            raise SvdqError(-2, "svdq_kv4_tree_attention")
        max_q, max_kv = _bound(max_q), _bound(max_kv)
        out = _empty((T, H, D), torch.bfloat16, dev, stream, Q) if out is None else _arg(
            out, torch.bfloat16, "out", (T, H, D))
        if lse is not None:
            _arg(lse, torch.float32, "lse", (T, H))
        if work is None:
            need = kv4_attention_workspace_bytes(cache, T, B, H, max_q, max_kv)
            work = _empty(need, torch.uint8, dev, stream) if need else None
        else:
            _arg(work, torch.uint8, "work")
        raw = _launch(dev, ("Q", "block_table", "q_start", "kv_len", "mask", "out", "lse", "work"),
                      (Q, block_table, q_start, kv_len, mask, out, lse, work), stream)
    st = lib().svdq_kv4_tree_attention(cache._ref, Q.data_ptr(), ldq, block_table.data_ptr(), width,
                                       q_start.data_ptr(), kv_len.data_ptr(), mask.data_ptr(), words, B, T, H, max_q,
                                       max_kv, D ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(lse),
                                       _ptr(work), 0 if work is None else work.numel(), raw)
    if st:
        raise SvdqError(st, "svdq_kv4_tree_attention")
    return out


TREE_MAX_WORDS = 32


def kv4_tree_plan(cache: Kv4Cache, parent, q_start, kv_len, block_table, max_q: int, mask=None, position=None,
                  slots=None, stream=None):
    """Mask, positions and slots of drafted tokens (one kernel): parent [T] int32,
    the number of each token's parent among its sequence's rows (smaller than its
    own; -1: a child of the last known token); max_q bounds the rows of a sequence
    (at most 1024) and gives the mask's words.  kv_len counts the drafted tokens.
    Returns (mask [T][ceil(max_q / 32)], position [T], slots [T]), int32."""
    torch = _T or _tt()
    raw = None
    try:
        T, = parent.shape
        B, width = block_table.shape
        dev = parent.get_device()
        if (stream is None and dev >= 0 and dev == _current_device() == cache.index == block_table.get_device()
                == q_start.get_device() == kv_len.get_device() and parent.dtype is _INT32 and block_table.dtype is _INT32
                and q_start.dtype is _INT32 and kv_len.dtype is _INT32 and q_start.shape == (B + 1,)
                and kv_len.shape == (B,) and parent.is_contiguous() and block_table.is_contiguous()
                and q_start.is_contiguous() and kv_len.is_contiguous() and 1 <= max_q <= 32 * TREE_MAX_WORDS
                and T < _I32 and B < _I32 and width < _I32):
            words = (max_q + 31) // 32
            if mask is None and position is None and slots is None:
                mask, position = parent.new_empty((T, words)), torch.empty_like(parent)
                slots = torch.empty_like(parent)
                raw = _raw_stream(dev)
    except _MISFIT:
        pass
    if raw is None:
        i32 = torch.int32
        dev = _cache_arg(cache)
        _ndim(parent, 1, "parent")
        _arg(parent, i32, "parent")
        T = parent.shape[0]
        _ndim(block_table, 2, "block_table")
        _arg(block_table, i32, "block_table")
        B, width = block_table.shape
        _arg(q_start, i32, "q_start", (B + 1,))
        _arg(kv_len, i32, "kv_len", (B,))
        if T > _I32 or B > _I32 or width > _I32:
            raise SvdqError(-2, "svdq_kv4_tree_plan")
        if not 1 <= max_q <= 32 * TREE_MAX_WORDS:
            raise ValueError(f"max_q must be 1 .. {32 * TREE_MAX_WORDS}, got {max_q}")
        words = (max_q + 31) // 32
        mask = _empty((T, words), i32, dev, stream) if mask is None else _arg(mask, i32, "mask", (T, words))
        position = _empty((T,), i32, dev, stream, parent) if position is None else _arg(position, i32, "position", (T,))
        slots = _empty((T,), i32, dev, stream, parent) if slots is None else _arg(slots, i32, "slots", (T,))
        raw = _launch(dev, ("parent", "q_start", "kv_len", "block_table", "mask", "position", "slots"),
                      (parent, q_start, kv_len, block_table, mask, position, slots), stream)
    st = lib().svdq_kv4_tree_plan(parent.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
                                  width, cache.pages, cache.page_size, B, T, mask.data_ptr(), words,
                                  position.data_ptr(), slots.data_ptr(), raw)
    if st:
        raise SvdqError(st, "svdq_kv4_tree_plan")
    return mask, position, slots


def kv4_keep_path(cache: Kv4Cache, path, q_start, kv_len, block_table, T: Optional[int] = None, new_len=None,
                  stream=None):
    """Moves the keys and values of each sequence's accepted rows, path [B][any]
    int32 (ascending, ended by -1), behind the known tokens (one kernel).  T: the
    step's rows; q_start's values are cut to it (None: not cut).  Returns the new
    lengths [B] int32 (not kv_len itself)."""
    torch = _T or _tt()
    raw = None
    try:
        B, longest = path.shape
        width, dev = block_table.shape[1], path.get_device()
        if (stream is None and new_len is None and T is None and dev >= 0
                and dev == _current_device() == cache.index == block_table.get_device() == q_start.get_device()
                == kv_len.get_device() and path.dtype is _INT32 and block_table.dtype is _INT32
                and q_start.dtype is _INT32 and kv_len.dtype is _INT32 and block_table.shape == (B, width)
                and q_start.shape == (B + 1,) and kv_len.shape == (B,) and path.is_contiguous()
                and block_table.is_contiguous() and q_start.is_contiguous() and kv_len.is_contiguous()
                and B < _I32 and longest < _I32 and width < _I32):
            new_len, T, raw = torch.empty_like(kv_len), _I32, _raw_stream(dev)
    except _MISFIT:
        pass
    if raw is None:
        i32 = torch.int32
        dev = _cache_arg(cache)
        _ndim(block_table, 2, "block_table")
        _arg(block_table, i32, "block_table")
        B, width = block_table.shape
        _ndim(path, 2, "path")
        longest = path.shape[1]
        _arg(path, i32, "path", (B, longest))
        _arg(q_start, i32, "q_start", (B + 1,))
        _arg(kv_len, i32, "kv_len", (B,))
        T = _I32 if T is None else max(T, -1)
        if B > _I32 or width > _I32 or longest > _I32 or T > _I32:
            raise SvdqError(-2, "svdq_kv4_keep_path")
        new_len = _empty((B,), i32, dev, stream, kv_len) if new_len is None else _arg(new_len, i32, "new_len", (B,))
        raw = _launch(dev, ("path", "q_start", "kv_len", "block_table", "new_len"),
                      (path, q_start, kv_len, block_table, new_len), stream)
    st = lib().svdq_kv4_keep_path(cache._ref, path.data_ptr(), longest, q_start.data_ptr(), kv_len.data_ptr(),
                                  block_table.data_ptr(), width, B, T, new_len.data_ptr(), raw)
    if st:
        raise SvdqError(st, "svdq_kv4_keep_path")
    return new_len


def rope_frequencies(sections, theta: float = 10000.0, layout: int = ROPE_AXES_BLOCKS):
    """Frequency (fp64) and axis (int32) of every pair of channels, for axes of
    `sections` pairs each (host, numpy)."""
    if np.ndim(sections) != 1:
        raise ValueError("sections must be one-dimensional")
    # what passes int32 stays too many, or negative, for the library to refuse
    sec = np.array([min(max(operator.index(n), -1), _I32) for n in sections], np.int32)
    n = int(sec.clip(0).sum(dtype=np.int64))
    freq, axis = np.empty(min(n, 128), np.float64), np.empty(min(n, 128), np.int32)
    _check(lib().svdq_rope_frequencies(sec.ctypes.data, sec.size, float(theta), layout, freq.ctypes.data,
                                       axis.ctypes.data), "svdq_rope_frequencies")
    return freq, axis


def rope_table(pos, freq, axis, cos=None, sin=None, stream=None):
    """cos and sin [T][pairs] fp32 of pos[t][axis[p]] * freq[p] (one kernel): pos
    [T][axes] int32, freq [pairs] fp64, axis [pairs] int32."""
    torch = _T or _tt()
    raw = None
    try:
        T, axes = pos.shape
        n, = freq.shape
        dev = pos.get_device()
        if (stream is None and cos is None and sin is None and dev >= 0
                and dev == _current_device() == freq.get_device() == axis.get_device() and pos.dtype is _INT32
                and axis.dtype is _INT32 and freq.dtype is _F64 and axis.shape == (n,) and pos.is_contiguous()
                and freq.is_contiguous() and axis.is_contiguous() and T < _I32 and axes < _I32 and n < _I32):
            cos = pos.new_empty((T, n), dtype=_F32)
            sin, raw = torch.empty_like(cos), _raw_stream(dev)
    except _MISFIT:
        pass
    if raw is None:
        f32 = torch.float32
        _ndim(pos, 2, "pos")
        _arg(pos, torch.int32, "pos")
        T, axes = pos.shape
        _ndim(freq, 1, "freq")
        _arg(freq, torch.float64, "freq")
        n = freq.shape[0]
        _arg(axis, torch.int32, "axis", (n,))
        if T > _I32 or axes > _I32 or n > _I32:
            raise SvdqError(-2, "svdq_rope_table")
        dev = pos.device
        cos = _empty((T, n), f32, dev, stream) if cos is None else _arg(cos, f32, "cos", (T, n))
        sin = _empty((T, n), f32, dev, stream, cos) if sin is None else _arg(sin, f32, "sin", (T, n))
        raw = _launch(dev, ("freq", "axis", "cos", "sin"), (freq, axis, cos, sin), stream)
    st = lib().svdq_rope_table(pos.data_ptr(), T, axes, freq.data_ptr(), axis.data_ptr(), n, cos.data_ptr(),
                               sin.data_ptr(), raw)
    if st:
        raise SvdqError(st, "svdq_rope_table")
    return cos, sin


def _rope_args(cos, sin, index, T, norm_q, norm_k, D):
    """Rows and pairs of the tables; checks what both rotating calls take."""
    torch = _T
    _ndim(cos, 2, "cos")
    _arg(cos, torch.float32, "cos")
    _arg(sin, torch.float32, "sin", cos.shape)
    if norm_q is not None:
        _arg(norm_q, torch.bfloat16, "norm_q", (D,))
    if norm_k is not None:
        _arg(norm_k, torch.bfloat16, "norm_k", (D,))
    if index is not None:
        _arg(index, torch.int32, "index", (T,))
    rows, pairs = cos.shape
    if rows > _I32 or pairs > _I32:
        raise ValueError("tables of more rows than the library takes")
    return rows, pairs


def _rope_fast(Q, K, V, Q_out, cos, sin, index, norm_q, norm_k):
    """Whether everything that both rotating calls take fits at once: the device and
    the row strides of Q, K, V and Q_out (V, Q_out may be None); else None."""
    T, H, D = Q.shape
    Hk, dev = K.shape[1], Q.get_device()
    ldq, hq, dq = Q.stride()
    ldk, hk, dk = K.stride()
    if not (dev >= 0 and dev == _current_device() == K.get_device() == cos.get_device() == sin.get_device()
            and Q.dtype is _BF and K.dtype is _BF and cos.dtype is _F32 and sin.dtype is _F32 and Hk
            and dq == 1 and dk == 1 and hq == D and hk == D and K.shape == (T, Hk, D) and cos.dim() == 2
            and cos.shape == sin.shape and cos.is_contiguous() and sin.is_contiguous() and 0 < T < _I32 > H
            and cos.shape[0] < _I32 and cos.shape[1] < _I32 and D < _I32 and Hk < _I32):
        return None
    for w in (norm_q, norm_k):
        if w is not None and not (w.dtype is _BF and w.shape == (D,) and w.get_device() == dev and w.is_contiguous()):
            return None
    if index is not None and not (index.dtype is _INT32 and index.shape == (T,) and index.get_device() == dev
                                  and index.is_contiguous()):
        return None
    ldv = ldo = H * D
    if V is not None:
        ldv, hv, dv = V.stride()
        if not (V.dtype is _BF and V.shape == (T, Hk, D) and dv == 1 and hv == D and V.get_device() == dev):
            return None
    if Q_out is not None:
        ldo, ho, do = Q_out.stride()
        if not (Q_out.dtype is _BF and Q_out.shape == (T, H, D) and do == 1 and ho == D and Q_out.get_device() == dev):
            return None
    if T == 1:                                          # a single row's stride does not matter
        ldq, ldk, ldv, ldo = H * D, Hk * D, Hk * D, H * D
    return dev, T, H, D, Hk, ldq, ldk, ldv, ldo


def qk_norm_rope(Q, K, cos, sin, style: int = ROPE_ADJACENT, index=None, norm_q=None, norm_k=None, eps: float = 1e-6,
                 Q_out=None, K_out=None, stream=None):
    """RMS-norm (with a weight norm_q, norm_k [dim]; None: no norm on that side)
    and rotation of query and key heads (one kernel).  Q [T][heads][dim], K
    [T][heads_k][dim] or None, bf16, dim 64, 128 or 256, rows may be a stride
    apart; cos, sin [rows][pairs] fp32 (rope_table), row of token t: index[t], or t;
    tokens without a row are not turned.  Q_out and K_out may be Q and K (in place).
    Returns (Q_out, K_out)."""
    torch = _T or _tt()
    raw = None
    if stream is None and Q_out is None and K_out is None:
        try:
            fit = _rope_fast(Q, K, None, None, cos, sin, index, norm_q, norm_k)
            if fit is not None:
                dev, T, H, D, Hk, ldq, ldk, _, ldqo = fit
                rows, pairs = cos.shape
                Q_out = torch.empty_like(Q) if ldq == H * D else Q.new_empty((T, H, D))      # like: 0.3 us less
                K_out = torch.empty_like(K) if ldk == Hk * D else K.new_empty((T, Hk, D))
                pK, pKo, ldko, raw = K.data_ptr(), K_out.data_ptr(), Hk * D, _raw_stream(dev)
        except _MISFIT:
            pass
    if raw is None:
        bf = torch.bfloat16
        _ndim(Q, 3, "Q")
        H, D = Q.shape[1:]
        T, ldq = _heads_arg(Q, "Q", H, D)
        rows, pairs = _rope_args(cos, sin, index, T, norm_q, norm_k, D)
        if T > _I32 or H > _I32 or D > _I32:
            raise SvdqError(-2, "svdq_qk_norm_rope")
        dev = Q.device
        if Q_out is None:
            Q_out = _empty((T, H, D), bf, dev, stream, Q)
        TO, ldqo = _heads_arg(Q_out, "Q_out", H, D)
        if TO != T:
            raise ValueError(f"Q_out has shape {tuple(Q_out.shape)}, expected {tuple(Q.shape)}")
        pK = pKo = None
        Hk = ldk = ldko = 0
        if K is not None:
            _ndim(K, 3, "K")
            Hk = K.shape[1]
            TK, ldk = _heads_arg(K, "K", Hk, D)
            if K_out is None:
                K_out = _empty((T, Hk, D), bf, dev, stream, K)
            TO, ldko = _heads_arg(K_out, "K_out", Hk, D)
            if TK != T or TO != T:
                raise ValueError("Q, K and K_out must have the same number of tokens")
            if Hk > _I32:
                raise SvdqError(-2, "svdq_qk_norm_rope")
            pK, pKo = K.data_ptr(), K_out.data_ptr()
        elif K_out is not None or norm_k is not None:
            raise ValueError("K_out or norm_k without K")
        raw = _launch(dev, ("K", "cos", "sin", "index", "norm_q", "norm_k", "Q_out", "K_out"),
                      (K, cos, sin, index, norm_q, norm_k, Q_out, K_out), stream)
    st = lib().svdq_qk_norm_rope(Q.data_ptr(), ldq, H, pK, ldk, Hk, T, D, _ptr(norm_q), _ptr(norm_k), eps,
                                 cos.data_ptr(), sin.data_ptr(), _ptr(index), rows, pairs, style, Q_out.data_ptr(),
                                 ldqo, pKo, ldko, raw)
    if st:
        raise SvdqError(st, "svdq_qk_norm_rope")
    return Q_out, K_out


def kv4_rope_append(cache: Kv4Cache, Q, K, V, cos, sin, slots, style: int = ROPE_ADJACENT, index=None, norm_q=None,
                    norm_k=None, eps: float = 1e-6, Q_out=None, stream=None):
    """qk_norm_rope on the way into the cache (one kernel): Q [T][heads][dim] to
    Q_out (may be Q), K and V [T][cache heads][dim] into their slots [T] int32, K
    normed and rotated first; the codes are those of qk_norm_rope and kv4_append.
    Returns Q_out."""
    torch = _T or _tt()
    raw = None
    if stream is None:
        try:
            fit = _rope_fast(Q, K, V, Q_out, cos, sin, index, norm_q, norm_k)
            if (fit is not None and V is not None and fit[0] == cache.index == slots.get_device() and fit[3] == cache.dim
                    and fit[4] == cache.heads and slots.dtype is _INT32 and slots.shape == (fit[1],)
                    and slots.is_contiguous()):
                dev, T, H, D, Hk, ldq, ldk, ldv, ldqo = fit
                rows, pairs = cos.shape
                if Q_out is None:
                    Q_out = torch.empty_like(Q) if ldq == H * D else Q.new_empty((T, H, D))
                raw = _raw_stream(dev)
        except _MISFIT:
            pass
    if raw is None:
        dev = _cache_arg(cache)
        Hk, D = cache.heads, cache.dim
        _ndim(Q, 3, "Q")
        H = Q.shape[1]
        T, ldq = _heads_arg(Q, "Q", H, D)
        TK, ldk = _heads_arg(K, "K", Hk, D)
        TV, ldv = _heads_arg(V, "V", Hk, D)
        if TK != T or TV != T:
            raise ValueError("Q, K and V must have the same number of tokens")
        _arg(slots, torch.int32, "slots", (T,))
        rows, pairs = _rope_args(cos, sin, index, T, norm_q, norm_k, D)
        if T > _I32 or H > _I32:
            raise SvdqError(-2, "svdq_kv4_rope_append")
        if Q_out is None:
            Q_out = _empty((T, H, D), torch.bfloat16, dev, stream, Q)
        TO, ldqo = _heads_arg(Q_out, "Q_out", H, D)
        if TO != T:
            raise ValueError(f"Q_out has shape {tuple(Q_out.shape)}, expected {tuple(Q.shape)}")
        raw = _launch(dev, ("Q", "K", "V", "cos", "sin", "slots", "index", "norm_q", "norm_k", "Q_out"),
                      (Q, K, V, cos, sin, slots, index, norm_q, norm_k, Q_out), stream)
    st = lib().svdq_kv4_rope_append(cache._ref, Q.data_ptr(), ldq, H, K.data_ptr(), V.data_ptr(), ldk, ldv,
                                    _ptr(norm_q), _ptr(norm_k), eps, cos.data_ptr(), sin.data_ptr(), _ptr(index),
                                    rows, pairs, style, slots.data_ptr(), T, Q_out.data_ptr(), ldqo, raw)
    if st:
        raise SvdqError(st, "svdq_kv4_rope_append")
    return Q_out


def to_device(packed: dict, device="cuda") -> dict:
    """Copy packed numpy arrays to device tensors with the dtypes the calls expect."""
    torch = _torch()
    out = {}
    for k, v in packed.items():
        t = torch.from_numpy(np.ascontiguousarray(v))
        if v.dtype == np.uint16:
            t = t.view(torch.int16).view(torch.bfloat16)
        out[k] = t.to(device)
    return out


def bf16_tensor(bits: np.ndarray, device="cuda"):
    """uint16 bf16 bits (numpy) -> torch bfloat16 tensor on `device`."""
    torch = _torch()
    return torch.from_numpy(np.ascontiguousarray(bits, np.uint16).view(np.int16)).view(
        torch.bfloat16).to(device)


def bf16_bits(t) -> np.ndarray:
    """torch bfloat16 tensor -> uint16 bits (numpy, host)."""
    torch = _torch()
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
