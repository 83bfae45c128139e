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

Device tensors: X bf16 [M][K], smooth fp32 [K], down bf16 [32][K],
up bf16 [N][32], bias bf16 [N] or None, xq uint8 [M][K/2],
xscale fp32 [M][K/64] (INT4) or uint8 [M][K/32] (MXFP4), h fp32 [M][32],
Y bf16 [M][N].  Calls are enqueued on the current torch stream (or `stream`).
"""
from __future__ import annotations

import ctypes
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
NORM_NONE = 0
NORM_RMS = 1
NORM_LAYER = 2
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
           "svdq_kv4_attention_workspace_bytes", "svdq_kv4_attention")


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


def _tt():
    global _T
    if _T is None:
        _T = _torch()
    return _T


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
