"""Refusals of the calls between the linears (residual + norm, adapters, 4-bit
cache): argument errors come back before the device is looked at, and the
binding checks every tensor against the shapes the call implies.  No GPU."""
import copy
import ctypes
import pickle

import numpy as np
import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
INVALID, SHAPE, MISALIGNED, UNSUPPORTED, DEVICE = -1, -2, -3, -4, -5
NO_GPU = not torch.cuda.is_available()


def _host(nbytes=1 << 12, offset=0):
    buf = np.zeros(nbytes + 64, np.uint8)
    return buf, buf.ctypes.data + (-buf.ctypes.data) % 16 + offset


_B1, P = _host()
_B2, Q = _host()
_B3, OFF = _host(offset=4)


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


# ------------------------------------------------------------- residual_norm

def _norm(**kw):
    a = dict(r=P, st=0, y=P, M=4, D=64, post=0, post_w=None, gate=None, alpha=1.0, pre=1, pre_w=None, pre_b=None,
             scale=None, shift=None, index=None, rows=0, stride=0, eps=1e-6, r_out=P, x=Q)
    a.update(kw)
    return svdq.lib().svdq_residual_norm(a["r"], a["st"], a["y"], a["M"], a["D"], a["post"], a["post_w"], a["gate"],
                                         a["alpha"], a["pre"], a["pre_w"], a["pre_b"], a["scale"], a["shift"],
                                         a["index"], a["rows"], a["stride"], a["eps"], a["r_out"], a["x"], None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(st=2)), (INVALID, dict(post=3)), (INVALID, dict(pre=-1)), (INVALID, dict(M=-1)),
    (INVALID, dict(eps=-1e-6)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(alpha=float("inf"))),
    (INVALID, dict(alpha=float("nan"))), (SHAPE, dict(D=60)), (SHAPE, dict(D=0)), (SHAPE, dict(D=16392)),
    (SHAPE, dict(M=1 << 24, D=64)), (INVALID, dict(r=None)), (INVALID, dict(r_out=None)), (INVALID, dict(x=P)),
    (INVALID, dict(r=Q, r_out=P, x=P)), (INVALID, dict(y=None)), (INVALID, dict(y=None, r_out=None, gate=P)),
    (INVALID, dict(y=None, r_out=None, x=None)), (INVALID, dict(gate=P, rows=0, stride=64)),
    (SHAPE, dict(scale=P, rows=2, stride=56)), (SHAPE, dict(scale=P, rows=2, stride=60)),
    (SHAPE, dict(scale=P, rows=3, stride=64)), (SHAPE, dict(shift=P, rows=1 << 15, stride=1 << 15, index=P)),
    (MISALIGNED, dict(r=OFF)), (MISALIGNED, dict(x=OFF)), (MISALIGNED, dict(gate=OFF, rows=1, stride=64)),
    (MISALIGNED, dict(gate=P, rows=1, stride=64, index=P + 2)), (MISALIGNED, dict(pre_w=OFF)),
])
def test_residual_norm_refusals(want, kw):
    assert _norm(**kw) == want


@pytest.mark.skipif(not NO_GPU, reason="checks the no-GPU path")
def test_accepted_arguments_reach_the_device_check():
    assert _norm() == DEVICE
    assert _norm(y=None, r_out=None) == DEVICE
    assert _norm(x=None) == DEVICE
    assert _norm(gate=P, rows=2, stride=64, index=P + 4) == DEVICE
    assert _norm(M=0, r=None, y=None, r_out=None, x=None) == DEVICE
    assert _plan() == _lora() == _append() == _read() == _attend() == DEVICE
    assert _lora(M=0, X=None, base=None, Y=None) == DEVICE
    assert _attend(T=0, Q=None, O=None) == DEVICE
    L = svdq.lib()
    assert L.svdq_lora_workspace_bytes(16, 64, 8, 2) == 0
    assert L.svdq_kv4_attention_workspace_bytes(_cache(), 16, 2, 4, 1, 100000) == 0


# ---------------------------------------------------------------------- lora

def _plan(index=P, M=16, n=4, plan=P, nbytes=None):
    L = svdq.lib()
    return L.svdq_lora_plan(index, M, n, plan, L.svdq_lora_plan_bytes(M, n) if nbytes is None else nbytes, None)


def _lora(**kw):
    a = dict(X=P, A=P, B=P, s=P, plan=P, base=P, M=16, N=64, K=64, R=8, n=4, Y=Q, work=P, wb=1 << 30)
    a.update(kw)
    return svdq.lib().svdq_lora_linear(a["X"], a["A"], a["B"], a["s"], a["plan"], a["base"], a["M"], a["N"], a["K"],
                                       a["R"], a["n"], a["Y"], a["work"], a["wb"], None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(N=-8)), (INVALID, dict(K=-8)), (SHAPE, dict(N=60)), (SHAPE, dict(K=60)),
    (SHAPE, dict(K=0)), (UNSUPPORTED, dict(R=0)), (UNSUPPORTED, dict(R=12)), (UNSUPPORTED, dict(R=136)),
    (UNSUPPORTED, dict(n=0)), (UNSUPPORTED, dict(n=4097)), (SHAPE, dict(M=1 << 20, K=1 << 10)),
    (SHAPE, dict(M=1 << 20, N=1 << 10)), (SHAPE, dict(n=4096, N=1 << 15)), (SHAPE, dict(n=4096, K=1 << 15)),
    (INVALID, dict(X=None)), (INVALID, dict(A=None)), (INVALID, dict(B=None)), (INVALID, dict(s=None)),
    (INVALID, dict(plan=None)), (INVALID, dict(base=None)), (INVALID, dict(Y=None)), (INVALID, dict(work=None)),
    (MISALIGNED, dict(X=OFF)), (MISALIGNED, dict(plan=OFF)), (MISALIGNED, dict(work=OFF)),
])
def test_lora_refusals(want, kw):
    assert _lora(**kw) == want


def test_lora_plan_refusals_and_sizes():
    L = svdq.lib()
    assert _plan(M=-1, nbytes=0) == INVALID
    assert _plan(n=0, nbytes=0) == UNSUPPORTED and _plan(n=4097, nbytes=0) == UNSUPPORTED
    assert _plan(index=None) == INVALID and _plan(plan=None) == INVALID
    assert _plan(nbytes=L.svdq_lora_plan_bytes(16, 4) - 1) == INVALID
    assert _plan(index=P + 2) == MISALIGNED and _plan(plan=OFF) == MISALIGNED
    assert L.svdq_lora_plan_bytes(0, 4) == L.svdq_lora_plan_bytes(16, 0) == 0
    # a header, then 64 places and 4 words for each of the tiles (at most one per row)
    assert L.svdq_lora_plan_bytes(1000, 7) == 4 * (16 + 68 * (1000 // 64 + 8))
    assert L.svdq_lora_plan_bytes(3, 4096) == 4 * (16 + 68 * 3)


def test_lora_binding_checks():
    M, K, N, R, n = 6, 64, 40, 8, 3
    plan = svdq.LoraPlan(z(4096, dtype=U8), M, n)
    good = dict(X=z(M, K), A=z(n, R, K), B=z(n, N, R), scale=z(n, dtype=F32), plan=plan, base=z(M, N))
    for name, bad in (("X", z(M, K, dtype=F32)), ("A", z(n, R, K, dtype=F32)), ("B", z(n, N, R, dtype=torch.float16)),
                      ("scale", z(n)), ("base", z(M, N, dtype=F32)), ("plan", z(8, dtype=U8)), ("X", [1])):
        with pytest.raises((TypeError, ValueError)):
            svdq.lora_linear(**dict(good, **{name: bad}), work=z(64, dtype=U8))
    for name, bad in (("A", z(n, R, K + 8)), ("B", z(n, N + 8, R)), ("B", z(n + 1, N, R)), ("scale", z(n + 1, dtype=F32)),
                      ("base", z(M + 1, N)), ("X", z(K, M).t()), ("base", z(M, 2 * N)[:, :N]),
                      ("plan", svdq.LoraPlan(plan.buffer, M + 1, n)), ("plan", svdq.LoraPlan(plan.buffer, M, n + 1))):
        with pytest.raises(ValueError):
            svdq.lora_linear(**dict(good, **{name: bad}), work=z(64, dtype=U8))
    with pytest.raises(ValueError, match="Y"):
        svdq.lora_linear(**good, Y=z(M, N + 8), work=z(64, dtype=U8))
    with pytest.raises(TypeError, match="device"):
        svdq.lora_linear(**good, Y=z(M, N), work=z(64, dtype=U8))
    with pytest.raises(TypeError, match="index"):
        svdq.lora_plan(z(4, dtype=torch.int64), 2)
    with pytest.raises(ValueError, match="plan"):
        svdq.lora_plan(z(M + 1, dtype=I32), n, plan=plan)


def test_residual_norm_binding_checks():
    M, D = 6, 64
    good = dict(r=z(M, D), y=z(M, D), gate=z(2, D), scale=z(2, D), shift=z(2, D))
    for name, bad in (("r", z(M, D, dtype=torch.float16)), ("y", z(M, D, dtype=F32)), ("gate", z(2, D, dtype=F32)),
                      ("mod_index", z(M, dtype=torch.int64)), ("pre_w", z(D, dtype=F32))):
        with pytest.raises(TypeError):
            svdq.residual_norm(**dict(good, **{name: bad}))
    for name, bad in (("y", z(M + 1, D)), ("gate", z(3, D)), ("scale", z(2, D + 8)), ("shift", z(D)), ("post_w", z(D + 8)),
                      ("mod_index", z(M + 1, dtype=I32)), ("r_out", z(M, D + 8)), ("x", z(M + 1, D)),
                      ("gate", z(2, 2 * D)[:, ::2]), ("gate", z(2, 2 * D)[:, :D]), ("gate", z(0, D)),
                      ("y", z(D, M).t()), ("r", z(M * D))):
        with pytest.raises(ValueError):
            svdq.residual_norm(**dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        svdq.residual_norm(z(M, D), r_out=z(M, D))
    with pytest.raises(ValueError):
        svdq.residual_norm(z(M, D), z(M, D), x=z(M, D), want_x=False)
    with pytest.raises(TypeError, match="device"):
        svdq.residual_norm(**good)


def test_broadcast_modulation_rows_are_refused():
    """An expanded vector has a row stride of 0: refused, not read past its end."""
    assert _norm(gate=P, rows=2, stride=0, index=P) == SHAPE


# ----------------------------------------------------------------------- kv4

def _cache(**kw):
    a = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, pages=4, page_size=16, heads=2, dim=64, prec=0)
    a.update(kw)
    c = svdq._Kv4Struct(*(a[f] for f, _ in svdq._Kv4Struct._fields_))
    _cache.keep = c
    return ctypes.addressof(c)


def _append(c=None, K=P, V=P, ldk=128, ldv=128, slots=P, T=8):
    return svdq.lib().svdq_kv4_append(_cache() if c is None else c, K, V, ldk, ldv, slots, T, None)


def _read(c=None, slots=P, T=8, K=P, V=P):
    return svdq.lib().svdq_kv4_read(_cache() if c is None else c, slots, T, K, V, None)


def _attend(c=None, **kw):
    a = dict(Q=P, ldq=256, table=P, width=2, start=P, kv=P, B=2, T=8, H=4, mq=1, mk=30, scale=0.125, causal=1, window=0,
             O=Q, lse=None, work=None, wb=0)
    a.update(kw)
    return svdq.lib().svdq_kv4_attention(_cache() if c is None else c, a["Q"], a["ldq"], a["table"], a["width"],
                                         a["start"], a["kv"], a["B"], a["T"], a["H"], a["mq"], a["mk"], a["scale"],
                                         a["causal"], a["window"], a["O"], a["lse"], a["work"], a["wb"], None)


CACHES = [(INVALID, dict(prec=2)), (INVALID, dict(pages=0)), (INVALID, dict(heads=0)), (UNSUPPORTED, dict(dim=96)),
          (UNSUPPORTED, dict(page_size=0)), (UNSUPPORTED, dict(page_size=8)), (UNSUPPORTED, dict(page_size=48)),
          (UNSUPPORTED, dict(page_size=512)), (UNSUPPORTED, dict(page_size=-16)), (SHAPE, dict(heads=65536)),
          (SHAPE, dict(pages=1 << 27)), (INVALID, dict(k_codes=None)), (INVALID, dict(v_scales=None)),
          (MISALIGNED, dict(v_codes=OFF)), (MISALIGNED, dict(k_scales=OFF))]


@pytest.mark.parametrize("want,kw", CACHES)
def test_cache_refusals(want, kw):
    assert _append(_cache(**kw)) == want
    assert _read(_cache(**kw)) == want
    assert _attend(_cache(**kw)) == want
    assert svdq.lib().svdq_kv4_attention_workspace_bytes(_cache(**kw), 8, 2, 4, 1, 30) == 0


def test_kv4_refusals():
    assert svdq.lib().svdq_kv4_append(None, P, P, 128, 128, P, 8, None) == INVALID
    for want, kw in ((INVALID, dict(T=-1)), (SHAPE, dict(T=1 << 24)), (SHAPE, dict(ldk=120)), (SHAPE, dict(ldv=132)),
                     (SHAPE, dict(ldk=1 << 40)), (INVALID, dict(K=None)), (INVALID, dict(slots=None)),
                     (MISALIGNED, dict(V=OFF)), (MISALIGNED, dict(slots=P + 1))):
        assert _append(**kw) == want, kw
    for want, kw in ((INVALID, dict(T=-1)), (SHAPE, dict(T=1 << 24)), (INVALID, dict(V=None)), (MISALIGNED, dict(K=OFF))):
        assert _read(**kw) == want, kw
    for want, kw in ((INVALID, dict(T=-1)), (INVALID, dict(B=-1)), (INVALID, dict(H=0)), (SHAPE, dict(H=3)),
                     (INVALID, dict(mq=0)), (INVALID, dict(mk=0)), (SHAPE, dict(T=1 << 23)), (SHAPE, dict(B=1 << 24)),
                     (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=float("nan"))),
                     (INVALID, dict(scale=float("inf"))), (INVALID, dict(scale=2.1e38)), (INVALID, dict(causal=2)), (INVALID, dict(window=-1)),
                     (INVALID, dict(causal=0, window=3)), (SHAPE, dict(ldq=248)), (SHAPE, dict(ldq=260)),
                     (INVALID, dict(width=0)), (SHAPE, dict(width=1 << 27)), (INVALID, dict(Q=None)),
                     (INVALID, dict(table=None)), (INVALID, dict(start=None)), (INVALID, dict(kv=None)),
                     (INVALID, dict(O=None)), (MISALIGNED, dict(Q=OFF)), (MISALIGNED, dict(table=P + 2)),
                     (MISALIGNED, dict(lse=OFF)), (MISALIGNED, dict(work=OFF))):
        assert _attend(**kw) == want, kw


def test_kv4_binding_checks():
    c = svdq.Kv4Cache(4, 16, 2, 64, svdq.INT4, device="cpu")
    assert c.k_codes.numel() == c.v_codes.numel() == 4 * 2 * 16 * 32 and c.k_scales.dtype is F32
    assert svdq.Kv4Cache(4, 16, 2, 64, svdq.MXFP4, device="cpu").v_scales.numel() == 4 * 2 * 16 * 2
    for kw in (dict(pages=0), dict(page_size=24), dict(heads=0), dict(dim=32), dict(prec=5),
               dict(pages=1 << 27), dict(heads=65536)):
        with pytest.raises(ValueError):
            svdq.Kv4Cache(**dict(dict(pages=4, page_size=16, heads=2, dim=64, prec=0, device="cpu"), **kw))
    K, s = z(5, 2, 64), z(5, dtype=I32)
    for bad in ((z(5, 3, 64), K, s), (K, z(5, 2, 128), s), (K, z(4, 2, 64), s), (K, K, z(4, dtype=I32)),
                (K.transpose(1, 2).contiguous().transpose(1, 2), K, s), (z(5, 4, 64)[:, ::2], K, s)):
        with pytest.raises(ValueError):
            svdq.kv4_append(c, *bad)
    for bad in ((z(5, 2, 64, dtype=F32), K, s), (K, K, z(5, dtype=torch.int64))):
        with pytest.raises(TypeError):
            svdq.kv4_append(c, *bad)
    with pytest.raises(TypeError, match="Kv4Cache"):
        svdq.kv4_append(None, K, K, s)
    with pytest.raises(TypeError, match="device"):
        svdq.kv4_append(c, K, K, s)
    with pytest.raises(TypeError, match="device"):
        svdq.kv4_read(c, s)
    good = dict(Q=z(5, 4, 64), cache=c, block_table=z(2, 3, dtype=I32), q_start=z(3, dtype=I32), kv_len=z(2, dtype=I32),
                max_q=1, max_kv=9, work=z(16, dtype=U8))
    for name, bad in (("Q", z(5, 3, 64)), ("Q", z(5, 4, 128)), ("Q", z(5, 256)), ("Q", z(5, 0, 64)),
                      ("block_table", z(6, dtype=I32)), ("q_start", z(2, dtype=I32)), ("kv_len", z(3, dtype=I32)),
                      ("block_table", z(3, 2, dtype=I32).t()), ("out", z(5, 4, 128)), ("lse", z(5, 5, dtype=F32))):
        with pytest.raises(ValueError):
            svdq.kv4_attention(**dict(good, **{name: bad}))
    for name, bad in (("Q", z(5, 4, 64, dtype=F32)), ("kv_len", z(2, dtype=torch.int64)), ("lse", z(5, 4)),
                      ("work", z(16, dtype=F32))):
        with pytest.raises(TypeError):
            svdq.kv4_attention(**dict(good, **{name: bad}))
    with pytest.raises(TypeError, match="device"):
        svdq.kv4_attention(**good)


def test_a_cache_is_not_copied():
    """A copy would hold the first cache's addresses."""
    c = svdq.Kv4Cache(1, 16, 1, 64, device="cpu")
    for f in (copy.copy, copy.deepcopy, pickle.dumps):
        with pytest.raises(TypeError):
            f(c)
