"""Rotary positions with several axes: the tables and the norm and rotation of
heads against their formulas in 64 bits, the form that appends to the 4-bit
cache against the two calls that it stands for, bit for bit.

Tolerances.  A table's value is the cosine or sine of the 64-bit product,
rounded once to fp32 (2^-24 relative); the product reduced by multiples of pi /
2 and the series add at most 2^-50 of 1 plus 2^-53 of the multiple.  A key's
value is computed in 64 bits from the same tables and rounded to fp32 and then
to bf16: 2^-24 + 2^-8 relative of the result, and of the pair's terms some
2^-50 (the formula's own roundings in another order).  A query's is fp32, u =
2^-24: the sum of 16 squares and up to four more sums is off by 20 u, its inverse
root by half of that and 3 u of its own (the mean with eps, the instruction), the
norm's two products by 2 u, the pair's by 2 u: 17 u of the pair's terms, called
20."""
import math
import sys

import numpy as np
import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
PRECS = [svdq.INT4, svdq.MXFP4]
STYLES = [svdq.ROPE_ADJACENT, svdq.ROPE_HALVES]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    x[..., ::13] *= 6.0
    return x.to(BF).cuda()


def _weight(seed, D):
    return (1.0 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(seed))).to(BF).cuda()


def _tables(seed, rows, pairs):
    a = 100.0 * torch.rand(rows, pairs, generator=torch.Generator().manual_seed(seed), dtype=F64)
    return a.cos().to(F32).cuda(), a.sin().to(F32).cuda()


def _formula(x, w, cos, sin, rows, style, eps):
    """The definition in 64 bits; rows [T], a value outside the tables does not turn.  Also the terms' magnitude."""
    u = x.to(F64)
    if w is not None:
        u = u / torch.sqrt((u ** 2).mean(-1, keepdim=True) + eps) * w.to(F64)
    n = cos.shape[1]
    ok = (rows >= 0) & (rows < cos.shape[0])
    at = torch.where(ok, rows, 0).long()
    c = torch.where(ok[:, None], cos.to(F64)[at], 1.0)[:, None]
    s = torch.where(ok[:, None], sin.to(F64)[at], 0.0)[:, None]
    o, mag = u.clone(), u.abs()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if style == svdq.ROPE_ADJACENT else (slice(0, n), slice(n, 2 * n))
    o[..., a], o[..., b] = u[..., a] * c - u[..., b] * s, u[..., b] * c + u[..., a] * s
    mag[..., a], mag[..., b] = (u[..., a] * c).abs() + (u[..., b] * s).abs(), (u[..., b] * c).abs() + (u[..., a] * s).abs()
    return o, mag


def _close(got, want, mag, key=False):
    lim = (2.0 ** -8 + 2.0 ** -24) * want.abs() + (2.0 ** -50 if key else 20 * 2.0 ** -24) * mag + 2.0 ** -133
    bad = (got.to(F64) - want).abs() > lim
    assert not bool(bad.any()), (int(bad.sum()), float(((got.to(F64) - want).abs() - lim).max()))


# ---------------------------------------------------------------------- tables

@pytest.mark.parametrize("T,sections,layout", [
    (1, (64,), svdq.ROPE_AXES_BLOCKS), (7, (8,), svdq.ROPE_AXES_SECTIONS), (333, (8, 28, 28), svdq.ROPE_AXES_BLOCKS),
    (1000, (16, 24, 24), svdq.ROPE_AXES_SECTIONS), (65, (24, 20, 20), svdq.ROPE_AXES_INTERLEAVED),
    (3, (0, 5, 40, 3, 80), svdq.ROPE_AXES_BLOCKS)])
def test_tables(T, sections, layout):
    _say(f"rope_table T={T} {sections} {layout}")
    freq, axis = svdq.rope_frequencies(sections, 10000.0, layout)
    g = np.random.default_rng(T)
    pos = g.integers(-2000, 100000, (T, len(sections)), dtype=np.int32)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = 2 ** 30, -2 ** 30 + 1
    cos, sin = svdq.rope_table(torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), torch.from_numpy(axis).cuda())
    angle = pos[:, axis].astype(np.float64) * freq
    for got, want in ((cos, np.cos(angle)), (sin, np.sin(angle))):
        d = np.abs(got.cpu().numpy().astype(np.float64) - want)
        assert (d <= 2.0 ** -24 * np.abs(want) + 2.0 ** -50 + 2.0 ** -53 * np.abs(angle) * 2 ** -50).all(), d.max()
    assert bool((cos[0] == 1).all()) and bool((sin[0] == 0).all())


def test_axes_outside_do_not_turn():
    pos = torch.full((4, 2), 17, dtype=I32, device="cuda")
    freq = torch.full((16,), 0.5, dtype=F64, device="cuda")
    axis = torch.tensor([0, 1, 2, -1, 2 ** 31 - 1, -2 ** 31, 1, 0] * 2, dtype=I32, device="cuda")
    cos, sin = svdq.rope_table(pos, freq, axis)
    turned = (axis == 0) | (axis == 1)
    assert bool((cos[:, turned] == torch.tensor(math.cos(8.5), dtype=F64).float()).all())
    assert bool((cos[:, ~turned] == 1).all()) and bool((sin[:, ~turned] == 0).all())


# -------------------------------------------------------------------- rotation

@pytest.mark.parametrize("style", STYLES)
@pytest.mark.parametrize("D,pairs", [(64, 32), (64, 8), (64, 16), (128, 64), (128, 24), (128, 32), (256, 128), (256, 64),
                                     (256, 40)])
@pytest.mark.parametrize("T,H,Hk", [(1, 1, 0), (1, 32, 8), (5, 7, 3), (700, 24, 24)])
def test_norm_and_rotation(style, D, pairs, T, H, Hk):
    _say(f"qk_norm_rope style={style} D={D} pairs={pairs} T={T} H={H} Hk={Hk}")
    Q = _rand(1, T, H, D)
    K = _rand(2, T, Hk, D) if Hk else None
    wq, wk = _weight(3, D), _weight(4, D) if Hk else None
    cos, sin = _tables(5, T, pairs)
    rows = torch.arange(T, device="cuda")
    q, k = svdq.qk_norm_rope(Q, K, cos, sin, style=style, norm_q=wq, norm_k=wk, eps=1e-5)
    _close(q, *_formula(Q, wq, cos, sin, rows, style, 1e-5))
    if Hk:
        _close(k, *_formula(K, wk, cos, sin, rows, style, 1e-5), key=True)
    q, k = svdq.qk_norm_rope(Q, K, cos, sin, style=style, norm_k=wk)        # the queries turned alone
    _close(q, *_formula(Q, None, cos, sin, rows, style, 0.0))
    if Hk:
        _close(k, *_formula(K, wk, cos, sin, rows, style, 1e-6), key=True)


@pytest.mark.parametrize("style", STYLES)
def test_strides_index_and_in_place(style):
    """Slices of a QKV product, rows of the tables by an index with values outside, outputs over the inputs."""
    T, H, Hk, D = 90, 5, 2, 128
    qkv = _rand(6, T, (H + 2 * Hk) * D)
    Q, K, V = (t.unflatten(1, (-1, D)) for t in qkv.split((H * D, Hk * D, Hk * D), 1))
    cos, sin = _tables(7, 40, 64)
    index = torch.randint(0, 40, (T,), generator=torch.Generator().manual_seed(1)).to(I32).cuda()
    index[3], index[4], index[5], index[6] = -1, 40, 2 ** 31 - 1, -2 ** 31
    w = _weight(8, D)
    wantq, wantk = _formula(Q, w, cos, sin, index, style, 1e-6), _formula(K, None, cos, sin, index, style, 0)
    before = V.clone()
    q, k = svdq.qk_norm_rope(Q, K, cos, sin, style=style, index=index, norm_q=w)
    _close(q, *wantq)
    _close(k, *wantk, key=True)
    q2, k2 = svdq.qk_norm_rope(Q, K, cos, sin, style=style, index=index, norm_q=w, Q_out=Q, K_out=K)
    assert q2 is Q and torch.equal(Q, q) and torch.equal(K, k) and torch.equal(V, before)
    # tokens past the tables, without an index
    q, _ = svdq.qk_norm_rope(V, None, cos, sin, style=style)
    _close(q, *_formula(V, None, cos, sin, torch.arange(T, device="cuda"), style, 0))
    assert torch.equal(q[40:], V[40:])


def test_values_far_apart():
    """Rows of zeros, of one value, of the type's largest and smallest."""
    D, T = 64, 6
    x = torch.zeros(T, 1, D, dtype=BF, device="cuda")
    x[1, 0, 5] = 3.0
    x[2] = 3e38
    x[3] = -1e-38
    x[4] = _rand(1, 1, D)[0] * 2.0 ** 100
    x[5] = _rand(2, 1, D)[0] * 2.0 ** -100
    cos, sin = _tables(9, T, 32)
    w = _weight(1, D)
    rows = torch.arange(T, device="cuda")
    for eps in (1e-6, 1e-30):
        q, _ = svdq.qk_norm_rope(x, None, cos, sin, norm_q=w, eps=eps)
        _close(q, *_formula(x, w, cos, sin, rows, svdq.ROPE_ADJACENT, eps))
        _, k = svdq.qk_norm_rope(x, x, cos, sin, norm_k=w, eps=eps)
        _close(k, *_formula(x, w, cos, sin, rows, svdq.ROPE_ADJACENT, eps), key=True)
    assert bool((q[0] == 0).all()) and bool((k[0] == 0).all())


@pytest.mark.parametrize("style", STYLES)
def test_infinite_values(style):
    """A head with an infinity: 1 / sqrt(inf) = 0, so its finite values become 0 and its infinity, and what that is
    rotated with, no number; other heads are as ever."""
    D, T = 128, 4
    x = _rand(1, T, 6, D)
    x[2, 3, 7] = math.inf
    x[3, 0, 9] = -math.inf
    cos, sin = _tables(9, T, D // 2)
    w = _weight(1, D)
    q, k = svdq.qk_norm_rope(x, x, cos, sin, style=style, norm_q=w, norm_k=w)
    clean = torch.where(torch.isinf(x), torch.zeros_like(x), x)
    wantq, wantk = svdq.qk_norm_rope(clean, clean, cos, sin, style=style, norm_q=w, norm_k=w)
    for got, want in ((q, wantq), (k, wantk)):
        for t, h, d in ((2, 3, 7), (3, 0, 9)):
            bad = torch.zeros(D, dtype=torch.bool, device="cuda")
            bad[d] = bad[d ^ 1 if style == svdq.ROPE_ADJACENT else (d + D // 2) % D] = True
            assert torch.equal(torch.isnan(got[t, h]), bad) and bool((got[t, h][~bad] == 0).all())
            want[t, h] = got[t, h] = 0
        assert torch.equal(got, want)


# ---------------------------------------------------------- on into the cache

@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("style", STYLES)
@pytest.mark.parametrize("D,pairs", [(64, 32), (64, 8), (128, 64), (128, 24)])
@pytest.mark.parametrize("T,H,Hk,P,norm", [(1, 8, 2, 16, True), (37, 12, 3, 32, True), (300, 4, 4, 256, False)])
def test_append_is_the_two_calls(prec, style, D, pairs, T, H, Hk, P, norm):
    _say(f"kv4_rope_append prec={prec} style={style} D={D} pairs={pairs} T={T} H={H} Hk={Hk} P={P}")
    qkv = _rand(T, T, (H + 2 * Hk) * D)
    Q, K, V = (t.unflatten(1, (-1, D)) for t in qkv.split((H * D, Hk * D, Hk * D), 1))
    cos, sin = _tables(11, T + 3, pairs)
    index = torch.randperm(T + 3, generator=torch.Generator().manual_seed(2))[:T].to(I32).cuda()
    wq, wk = (_weight(1, D), _weight(2, D)) if norm else (None, None)
    pages = -(-T // P) + 2
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(T))[:T].to(I32).cuda()
    if T > 20:
        slots[5], slots[17] = -1, pages * P
    caches = [svdq.Kv4Cache(pages, P, Hk, D, prec) for _ in range(2)]
    for c in caches:
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            t.view(torch.uint8).fill_(255)
    q, k = svdq.qk_norm_rope(Q, K, cos, sin, style=style, index=index, norm_q=wq, norm_k=wk)
    svdq.kv4_append(caches[0], k, V, slots)
    got = svdq.kv4_rope_append(caches[1], Q, K, V, cos, sin, slots, style=style, index=index, norm_q=wq, norm_k=wk)
    assert torch.equal(got, q)
    for a, b in ((c.view(torch.uint8), d.view(torch.uint8)) for c, d in (
            (caches[0].k_codes, caches[1].k_codes), (caches[0].v_codes, caches[1].v_codes),
            (caches[0].k_scales, caches[1].k_scales), (caches[0].v_scales, caches[1].v_scales))):
        assert torch.equal(a, b)


def test_nothing_to_do():
    c = svdq.Kv4Cache(1, 16, 2, 64)
    cos, sin = _tables(1, 4, 32)
    e = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    k = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    assert svdq.qk_norm_rope(e, k, cos, sin)[1].shape == (0, 2, 64)
    assert svdq.kv4_rope_append(c, e, k, k, cos, sin, torch.empty(0, dtype=I32, device="cuda")).shape == e.shape
    none = torch.empty(0, 32, dtype=F32, device="cuda")
    q, _ = svdq.qk_norm_rope(_rand(1, 3, 4, 64), None, none, none)          # tables without rows: nothing turns
    assert torch.equal(q, _rand(1, 3, 4, 64))
    f = torch.ones(8, dtype=F64, device="cuda")
    cs, _ = svdq.rope_table(torch.empty(0, 1, dtype=I32, device="cuda"), f, torch.zeros(8, dtype=I32, device="cuda"))
    assert cs.shape == (0, 8)
