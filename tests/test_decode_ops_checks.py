"""Refusals of the decoding calls (rotary positions, drafted trees, linears of few
rows, gated linears): argument errors come back before the device is looked at,
and the binding checks every tensor against the shapes the call implies.  No
GPU."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")

BF, F32, F64, U8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.uint8, torch.int32
INVALID, SHAPE, MISALIGNED, UNSUPPORTED, DEVICE = -1, -2, -3, -4, -5
NO_GPU = not torch.cuda.is_available()
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _host(nbytes=1 << 12, offset=0):
    buf = np.zeros(nbytes + 64, np.uint8)
    return buf, buf.ctypes.data + (-buf.ctypes.data) % 16 + offset


_B1, P = _host()
_B2, Q = _host()
_B3, OFF = _host(offset=4)


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def _cache(pages=4, page=16, heads=2, dim=64, prec=svdq.INT4, base=None):
    b = P if base is None else base
    return ctypes.byref(svdq._Kv4Struct(b, b, b, b, pages, page, heads, dim, prec))


# -------------------------------------------------------------------- linears

def _linear(name, **kw):
    a = dict(xq=P, xs=P, h=P, wq=P, ws=P, up=P, bias=None, M=4, N=64, K=128, r=32, prec=svdq.INT4, last=0, Y=Q)
    a.update(kw)
    return getattr(svdq.lib(), name)(a["xq"], a["xs"], a["h"], a["wq"], a["ws"], a["up"], a["bias"], a["M"], a["N"],
                                     a["K"], a["r"], a["prec"], a["last"], a["Y"], None)


BOTH = ["svdq_w4a4_linear_few", "svdq_w4a4_linear_gated"]


@pytest.mark.parametrize("name", BOTH)
@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(N=-8)), (INVALID, dict(prec=2)), (INVALID, dict(last=2)),
    (INVALID, dict(last=-1)), (UNSUPPORTED, dict(r=16)), (SHAPE, dict(K=96)), (SHAPE, dict(K=0)), (SHAPE, dict(N=60)),
    (SHAPE, dict(N=1 << 24, K=128)), (SHAPE, dict(prec=svdq.MXFP4, K=48)), (INVALID, dict(xq=None)),
    (INVALID, dict(xs=None)), (INVALID, dict(h=None)), (INVALID, dict(wq=None)), (INVALID, dict(ws=None)),
    (INVALID, dict(up=None)), (INVALID, dict(Y=None)), (MISALIGNED, dict(xq=OFF)), (MISALIGNED, dict(bias=OFF)),
    (MISALIGNED, dict(Y=OFF)), (MISALIGNED, dict(h=OFF)), (MISALIGNED, dict(up=OFF)),
])
def test_linear_refusals(name, want, kw):
    assert _linear(name, **kw) == want


def test_linear_limits():
    assert _linear("svdq_w4a4_linear_few", M=svdq.FEW_MAX_ROWS + 1) == UNSUPPORTED
    # 2 F rows of the weight count
    assert _linear("svdq_w4a4_linear_gated", N=1 << 22, K=128) == SHAPE
    assert _linear("svdq_w4a4_linear_few", N=1 << 22, K=128) != SHAPE
    if NO_GPU:
        assert _linear("svdq_w4a4_linear_few", M=svdq.FEW_MAX_ROWS) == DEVICE
        assert _linear("svdq_w4a4_linear_gated", M=5000, prec=svdq.MXFP4, K=32, bias=P) == DEVICE
        assert _linear("svdq_w4a4_linear_few", M=0, xq=None, xs=None, h=None, Y=None) == DEVICE
        assert _linear("svdq_w4a4_linear_gated", N=0, wq=None, ws=None, up=None, Y=None) == DEVICE


@pytest.mark.parametrize("call,rows", [(svdq.w4a4_linear_few, 1), (svdq.w4a4_linear_gated, 2)])
@pytest.mark.parametrize("prec", [svdq.INT4, svdq.MXFP4])
def test_linear_binding_checks(call, rows, prec):
    M, N, K = 3, 16, 128
    g, sdt = svdq.group_of(prec), F32 if prec == svdq.INT4 else U8
    good = dict(xq=z(M, K // 2, dtype=U8), xscale=z(M, K // g, dtype=sdt), h=z(M, 32, dtype=F32),
                wq=z(rows * N, K // 2, dtype=U8), wscale=z(rows * N, K // g, dtype=sdt), up=z(rows * N, 32),
                bias=z(rows * N))
    for name, bad, err in (
            ("xq", z(M, K // 2, dtype=torch.int8), TypeError), ("xq", z(K // 2, dtype=U8), ValueError),
            ("xscale", z(M, K // g, dtype=U8 if prec == svdq.INT4 else F32), TypeError),
            ("xscale", z(M, K // g + 1, dtype=sdt), ValueError), ("h", z(M + 1, 32, dtype=F32), ValueError),
            ("h", z(M, 32), TypeError), ("wq", z(rows * N, K, dtype=U8), ValueError),
            ("wscale", z(N + 3, K // g, dtype=sdt), ValueError), ("up", z(rows * N, 32, dtype=F32), TypeError),
            ("up", z(32, rows * N).t(), ValueError), ("bias", z(N + 1), ValueError), ("bias", z(rows * N, dtype=F32), TypeError),
            ("Y", z(M, N + 8), ValueError), ("Y", z(M, N, dtype=F32), TypeError), ("Y", z(N, M).t(), ValueError),
            ("wq", None, ValueError), ("h", None, TypeError)):
        with pytest.raises(err):
            call(**{**good, name: bad}, prec=prec)
    with pytest.raises(ValueError):
        call(**good, prec=7)
    if rows == 2:
        with pytest.raises(ValueError):
            call(**{**good, "wq": z(33, K // 2, dtype=U8), "wscale": z(33, K // g, dtype=sdt), "up": z(33, 32),
                    "bias": None}, prec=prec)
    if NO_GPU:
        with pytest.raises(TypeError, match="device tensor"):
            call(**good, prec=prec)


# ------------------------------------------------------------------ positions

def _frequencies(sections, theta=10000.0, layout=0):
    sec = (ctypes.c_int * max(1, len(sections)))(*sections)
    f, a = (ctypes.c_double * 128)(), (ctypes.c_int32 * 128)()
    st = svdq.lib().svdq_rope_frequencies(sec, len(sections), theta, layout, f, a)
    return st, list(f), list(a)


def test_frequencies():
    """The layouts by their definition."""
    for sections in ((64,), (8, 28, 28), (16, 24, 24), (0, 8), (1, 2, 3, 2)):
        n = sum(sections)
        run = [a for a, k in enumerate(sections) for _ in range(k)]
        for theta in (10000.0, 1e6, 0.5):
            f, a = svdq.rope_frequencies(sections, theta, svdq.ROPE_AXES_BLOCKS)
            assert a.tolist() == run and f.dtype == np.float64 and a.dtype == np.int32
            assert np.allclose(f, [theta ** (-j / k) for k in sections for j in range(k)], rtol=1e-15, atol=0)
            f, a = svdq.rope_frequencies(sections, theta, svdq.ROPE_AXES_SECTIONS)
            assert a.tolist() == run and np.allclose(f, [theta ** (-p / n) for p in range(n)], rtol=1e-15, atol=0)
            f, a = svdq.rope_frequencies(sections, theta, svdq.ROPE_AXES_INTERLEAVED)
            k = len(sections)
            assert a.tolist() == [p % k if p // k < sections[p % k] else 0 for p in range(n)]
            assert np.allclose(f, [theta ** (-p / n) for p in range(n)], rtol=1e-15, atol=0)


def test_frequency_refusals():
    assert _frequencies((8,))[0] == 0
    for sections in ((4,), (12,), (136,), (), (0,), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert _frequencies(sections)[0] in (SHAPE, INVALID)
    assert _frequencies((16, -8))[0] == INVALID and _frequencies((1,) * 9)[0] == INVALID
    for theta in (0.0, -1.0, math.nan, math.inf):
        assert _frequencies((8,), theta)[0] == INVALID
    assert _frequencies((8,), layout=3)[0] == INVALID and _frequencies((8,), layout=-1)[0] == INVALID
    L = svdq.lib()
    assert L.svdq_rope_frequencies(None, 1, 1e4, 0, P, P) == INVALID
    for bad in ((4,), (-8, 16), (8, 8, 1)):
        with pytest.raises(svdq.SvdqError):
            svdq.rope_frequencies(bad)


def _table(**kw):
    a = dict(pos=P, T=4, axes=3, freq=P, axis=P, pairs=64, cos=P, sin=Q)
    a.update(kw)
    return svdq.lib().svdq_rope_table(a["pos"], a["T"], a["axes"], a["freq"], a["axis"], a["pairs"], a["cos"], a["sin"], None)


def _rotate(**kw):
    a = dict(Q=P, ldq=256, hq=4, K=P, ldk=128, hk=2, T=3, dim=64, wq=P, wk=None, eps=1e-6, cos=P, sin=P, index=None,
             rows=3, pairs=32, style=0, Qo=Q, ldqo=256, Ko=Q, ldko=128)
    a.update(kw)
    return svdq.lib().svdq_qk_norm_rope(a["Q"], a["ldq"], a["hq"], a["K"], a["ldk"], a["hk"], a["T"], a["dim"], a["wq"],
                                        a["wk"], a["eps"], a["cos"], a["sin"], a["index"], a["rows"], a["pairs"],
                                        a["style"], a["Qo"], a["ldqo"], a["Ko"], a["ldko"], None)


def _rope_append(**kw):
    a = dict(c=_cache(), Q=P, ldq=256, hq=4, K=P, V=P, ldk=128, ldv=128, wq=None, wk=P, eps=1e-6, cos=P, sin=P,
             index=None, rows=3, pairs=32, style=1, slots=P, T=3, Qo=Q, ldqo=256)
    a.update(kw)
    return svdq.lib().svdq_kv4_rope_append(a["c"], a["Q"], a["ldq"], a["hq"], a["K"], a["V"], a["ldk"], a["ldv"],
                                           a["wq"], a["wk"], a["eps"], a["cos"], a["sin"], a["index"], a["rows"],
                                           a["pairs"], a["style"], a["slots"], a["T"], a["Qo"], a["ldqo"], None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(T=-1)), (INVALID, dict(axes=0)), (INVALID, dict(axes=9)), (SHAPE, dict(pairs=4)),
    (SHAPE, dict(pairs=60)), (SHAPE, dict(pairs=136)), (SHAPE, dict(T=1 << 24)), (INVALID, dict(pos=None)),
    (INVALID, dict(freq=None)), (INVALID, dict(axis=None)), (INVALID, dict(cos=None)), (INVALID, dict(sin=None)),
    (MISALIGNED, dict(pos=P + 2)), (MISALIGNED, dict(freq=OFF)), (MISALIGNED, dict(axis=P + 1)),
    (MISALIGNED, dict(cos=OFF)),
])
def test_table_refusals(want, kw):
    assert _table(**kw) == want


@pytest.mark.parametrize("call", [_rotate, _rope_append])
@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(T=-1)), (INVALID, dict(hq=0)), (INVALID, dict(style=2)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=math.nan)), (INVALID, dict(eps=math.inf)), (INVALID, dict(rows=-1)), (SHAPE, dict(pairs=4)),
    (SHAPE, dict(pairs=40)), (SHAPE, dict(pairs=12)), (SHAPE, dict(ldq=248)), (SHAPE, dict(ldq=260)),
    (SHAPE, dict(ldk=120)), (SHAPE, dict(ldqo=8)), (SHAPE, dict(T=1 << 22)), (INVALID, dict(Q=None)),
    (INVALID, dict(K=None)), (INVALID, dict(Qo=None)), (INVALID, dict(cos=None)), (INVALID, dict(sin=None)),
    (INVALID, dict(Qo=P, ldqo=512)), (MISALIGNED, dict(Q=OFF)), (MISALIGNED, dict(K=OFF)), (MISALIGNED, dict(cos=OFF)),
    (MISALIGNED, dict(wk=OFF)), (MISALIGNED, dict(index=P + 2)), (MISALIGNED, dict(Qo=OFF)), (SHAPE, dict(hq=70000, ldq=1 << 23, ldqo=1 << 23)),
])
def test_rotation_refusals(call, want, kw):
    assert call(**kw) == want


def test_rotation_refusals_of_one_form():
    assert _rotate(dim=96) == UNSUPPORTED and _rotate(dim=32) == UNSUPPORTED and _rotate(hk=-1) == INVALID
    assert _rotate(Ko=None) == INVALID and _rotate(Ko=P, ldko=256) == INVALID and _rotate(ldko=64) == SHAPE
    assert _rope_append(V=None) == INVALID and _rope_append(slots=None) == INVALID and _rope_append(slots=P + 1) == MISALIGNED
    assert _rope_append(ldv=64) == SHAPE and _rope_append(V=OFF) == MISALIGNED
    assert _rope_append(c=_cache(page=24)) == UNSUPPORTED and _rope_append(c=_cache(dim=96)) == UNSUPPORTED
    assert _rope_append(c=_cache(prec=5)) == INVALID and _rope_append(c=_cache(base=OFF)) == MISALIGNED
    if NO_GPU:
        assert _table() == _rotate() == _rope_append() == DEVICE
        assert _rotate(K=None, Ko=None, hk=0, ldk=0, ldko=0) == DEVICE
        assert _rotate(Qo=P, Ko=P) == DEVICE                               # in place
        assert _rotate(T=0, Q=None, K=None, Qo=None, Ko=None) == DEVICE and _table(T=0, pos=None, cos=None, sin=None) == DEVICE
        assert _rotate(rows=0, cos=None, sin=None) == DEVICE


def test_rotation_binding_checks():
    T, H, Hk, D, n = 5, 4, 2, 64, 32
    cos, sin = z(T, n, dtype=F32), z(T, n, dtype=F32)
    good = dict(Q=z(T, H, D), K=z(T, Hk, D), cos=cos, sin=sin)
    for kw, err in ((dict(Q=z(T, H, D, dtype=F32)), TypeError), (dict(Q=z(T, H * D)), ValueError),
                    (dict(K=z(T + 1, Hk, D)), ValueError), (dict(K=z(T, Hk, 128)), ValueError),
                    (dict(Q=z(T, D, H).transpose(1, 2)), ValueError), (dict(cos=z(T, n)), TypeError),
                    (dict(sin=z(T, n + 8, dtype=F32)), ValueError), (dict(cos=z(n, T, dtype=F32).t()), ValueError),
                    (dict(norm_q=z(D, dtype=F32)), TypeError), (dict(norm_k=z(D + 1)), ValueError),
                    (dict(index=z(T, dtype=torch.int64)), TypeError), (dict(index=z(T + 1, dtype=I32)), ValueError),
                    (dict(Q_out=z(T, H, D, dtype=F32)), TypeError), (dict(Q_out=z(T + 1, H, D)), ValueError),
                    (dict(K_out=z(T, H, D)), ValueError), (dict(K=None, K_out=z(T, Hk, D)), ValueError),
                    (dict(K=None, norm_k=z(D)), ValueError), (dict(Q=[1]), ValueError), (dict(cos=None), ValueError), (dict(sin=None), TypeError)):
        with pytest.raises(err):
            svdq.qk_norm_rope(**{**good, **kw})
    c = svdq.Kv4Cache(2, 16, Hk, D, svdq.MXFP4, device="cpu")
    more = dict(good, cache=c, V=z(T, Hk, D), slots=z(T, dtype=I32))
    for kw, err in ((dict(V=z(T, Hk, D, dtype=F32)), TypeError), (dict(V=z(T - 1, Hk, D)), ValueError),
                    (dict(K=z(T, Hk + 1, D)), ValueError), (dict(slots=z(T, dtype=torch.int64)), TypeError),
                    (dict(slots=z(T - 1, dtype=I32)), ValueError), (dict(cache=None), TypeError),
                    (dict(Q=z(T, H, 128)), ValueError), (dict(Q_out=z(T, H, 128)), ValueError)):
        with pytest.raises(err):
            svdq.kv4_rope_append(**{**more, **kw})
    pos, freq, axis = z(T, 3, dtype=I32), z(n, dtype=F64), z(n, dtype=I32)
    for args, err in (((pos.long(), freq, axis), TypeError), ((pos[0], freq, axis), ValueError),
                      ((pos, freq.float(), axis), TypeError), ((pos, freq, axis[1:]), ValueError),
                      ((pos, freq, axis.long()), TypeError), ((pos.t(), freq, axis), ValueError)):
        with pytest.raises(err):
            svdq.rope_table(*args)
    with pytest.raises(ValueError):
        svdq.rope_table(pos, freq, axis, cos=z(T, n + 1, dtype=F32))
    if NO_GPU:
        for f in (lambda: svdq.qk_norm_rope(**good), lambda: svdq.kv4_rope_append(**more), lambda: svdq.rope_table(pos, freq, axis)):
            with pytest.raises(TypeError, match="device tensor"):
                f()


# ---------------------------------------------------------------------- trees

def _plan(**kw):
    a = dict(parent=P, qs=P, kl=P, table=P, width=4, pages=8, page=16, B=2, T=6, mask=Q, words=1, pos=Q, slots=Q)
    a.update(kw)
    return svdq.lib().svdq_kv4_tree_plan(a["parent"], a["qs"], a["kl"], a["table"], a["width"], a["pages"], a["page"],
                                         a["B"], a["T"], a["mask"], a["words"], a["pos"], a["slots"], None)


def _attend(**kw):
    a = dict(c=_cache(), Q=P, ldq=256, table=P, width=4, qs=P, kl=P, mask=P, words=1, B=2, T=6, hq=4, mq=3, mk=64,
             scale=0.1, O=Q, lse=None, work=P, wb=1 << 30)
    a.update(kw)
    return svdq.lib().svdq_kv4_tree_attention(a["c"], a["Q"], a["ldq"], a["table"], a["width"], a["qs"], a["kl"],
                                              a["mask"], a["words"], a["B"], a["T"], a["hq"], a["mq"], a["mk"],
                                              a["scale"], a["O"], a["lse"], a["work"], a["wb"], None)


def _keep(**kw):
    a = dict(c=_cache(), path=P, most=4, qs=P, kl=P, table=P, width=4, B=2, T=6, new=Q)
    a.update(kw)
    return svdq.lib().svdq_kv4_keep_path(a["c"], a["path"], a["most"], a["qs"], a["kl"], a["table"], a["width"],
                                         a["B"], a["T"], a["new"], None)


@pytest.mark.parametrize("call,want,kw", [
    (_plan, INVALID, dict(T=-1)), (_plan, INVALID, dict(B=-1)), (_plan, INVALID, dict(width=0)),
    (_plan, INVALID, dict(pages=0)), (_plan, UNSUPPORTED, dict(page=48)), (_plan, SHAPE, dict(pages=1 << 28)),
    (_plan, SHAPE, dict(width=1 << 28)), (_plan, SHAPE, dict(B=1 << 24)), (_plan, INVALID, dict(words=0)),
    (_plan, SHAPE, dict(words=33)), (_plan, SHAPE, dict(T=1 << 26, words=32)), (_plan, INVALID, dict(parent=None)),
    (_plan, INVALID, dict(mask=None)), (_plan, INVALID, dict(table=None)), (_plan, MISALIGNED, dict(parent=P + 1)),
    (_plan, MISALIGNED, dict(mask=P + 2)), (_plan, MISALIGNED, dict(pos=P + 2)), (_plan, MISALIGNED, dict(slots=P + 3)),
    (_attend, INVALID, dict(words=0)), (_attend, SHAPE, dict(words=33)), (_attend, INVALID, dict(mask=None)),
    (_attend, MISALIGNED, dict(mask=P + 2)), (_attend, INVALID, dict(B=-1)), (_attend, INVALID, dict(T=-1)),
    (_attend, SHAPE, dict(hq=3)), (_attend, INVALID, dict(mq=0)), (_attend, INVALID, dict(mk=0)),
    (_attend, INVALID, dict(scale=0.0)), (_attend, INVALID, dict(scale=math.nan)), (_attend, SHAPE, dict(ldq=64)),
    (_attend, INVALID, dict(Q=None)), (_attend, INVALID, dict(O=None)), (_attend, INVALID, dict(kl=None)),
    (_attend, MISALIGNED, dict(O=OFF)), (_attend, MISALIGNED, dict(lse=OFF)), (_attend, INVALID, dict(width=0)),
    (_attend, UNSUPPORTED, dict(c=_cache(dim=80))), (_keep, INVALID, dict(most=0)), (_keep, INVALID, dict(B=-1)),
    (_keep, INVALID, dict(T=-1)), (_keep, INVALID, dict(path=None)), (_keep, INVALID, dict(new=None)),
    (_keep, INVALID, dict(new=P)), (_keep, MISALIGNED, dict(path=P + 2)), (_keep, MISALIGNED, dict(new=Q + 2)),
    (_keep, SHAPE, dict(B=1 << 23)), (_keep, SHAPE, dict(B=1 << 20, most=1 << 10)), (_keep, UNSUPPORTED, dict(c=_cache(page=8))),
    (_keep, INVALID, dict(c=None)),
])
def test_tree_refusals(call, want, kw):
    assert call(**kw) == want


@pytest.mark.skipif(not NO_GPU, reason="checks the no-GPU path")
def test_accepted_trees_reach_the_device_check():
    assert _plan() == _attend() == _keep() == DEVICE
    assert _plan(pos=None, slots=None) == DEVICE and _plan(T=0, parent=None, mask=None) == DEVICE
    assert _attend(T=0, Q=None, O=None, mask=None) == DEVICE and _keep(B=0, path=None, new=None) == DEVICE


def test_tree_binding_checks():
    T, B, H, D = 6, 2, 4, 64
    c = svdq.Kv4Cache(4, 16, 2, D, svdq.INT4, device="cpu")
    parent, qs, kl, table = z(T, dtype=I32), z(B + 1, dtype=I32), z(B, dtype=I32), z(B, 3, dtype=I32)
    good = dict(cache=c, parent=parent, q_start=qs, kv_len=kl, block_table=table, max_q=4)
    for kw, err in ((dict(cache=1), TypeError), (dict(parent=parent.long()), TypeError), (dict(parent=z(2, 3, dtype=I32)), ValueError),
                    (dict(q_start=z(B, dtype=I32)), ValueError), (dict(kv_len=z(B + 1, dtype=I32)), ValueError),
                    (dict(block_table=z(B, dtype=I32)), ValueError), (dict(max_q=0), ValueError), (dict(max_q=1025), ValueError),
                    (dict(mask=z(T, 2, dtype=I32)), ValueError), (dict(position=z(T, dtype=F32)), TypeError),
                    (dict(slots=z(T + 1, dtype=I32)), ValueError)):
        with pytest.raises(err):
            svdq.kv4_tree_plan(**{**good, **kw})
    att = dict(Q=z(T, H, D), cache=c, block_table=table, q_start=qs, kv_len=kl, mask=z(T, 1, dtype=I32), max_q=4, max_kv=40)
    for kw, err in ((dict(mask=z(T, dtype=I32)), ValueError), (dict(mask=z(T + 1, 1, dtype=I32)), ValueError),
                    (dict(mask=z(T, 1, dtype=torch.int64)), TypeError), (dict(Q=z(T, 3, D)), ValueError),
                    (dict(Q=z(T, H, 128)), ValueError), (dict(out=z(T, H, D, dtype=F32)), TypeError),
                    (dict(lse=z(T, H)), TypeError), (dict(kv_len=z(B, dtype=F32)), TypeError)):
        with pytest.raises(err):
            svdq.kv4_tree_attention(**{**att, **kw})
    keep = dict(cache=c, path=z(B, 5, dtype=I32), q_start=qs, kv_len=kl, block_table=table)
    for kw, err in ((dict(path=z(B + 1, 5, dtype=I32)), ValueError), (dict(path=z(B, 5)), TypeError),
                    (dict(path=z(5, B, dtype=I32).t()), ValueError), (dict(new_len=z(B + 1, dtype=I32)), ValueError),
                    (dict(block_table=table.long()), TypeError)):
        with pytest.raises(err):
            svdq.kv4_keep_path(**{**keep, **kw})
    if NO_GPU:
        for f in (lambda: svdq.kv4_tree_plan(**good), lambda: svdq.kv4_tree_attention(**att, work=z(16, dtype=U8)),
                  lambda: svdq.kv4_keep_path(**keep)):
            with pytest.raises(TypeError, match="device tensor"):
                f()


def test_tree_attention_launches(tmp_path):
    """Every launch that the size checks let through is one that the runtime takes, and fits the workspace."""
    exe = str(tmp_path / "check")
    csrc = os.path.join(ROOT, "w4a4_rank_corrected_quantize_amd", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, os.path.join(ROOT, "tests", "native", "kv4_tree_plan_check.cpp"),
                    "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
