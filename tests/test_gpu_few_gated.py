"""The 4-bit linear of few rows and the gated linear against the formula in 64
bits over the decoded codes.

Bound, u = 2^-24, S = sum_k |x w| of an output, L = sum_j |h up|.  A group's or
block's products are exact and their sum is one of fp32 (INT4: exact), so the
4-bit term is off by at most (K + 8) u S, plus the scales' product: u S (few
rows, MXFP4: exact) or 2^-15 S (the INT4 tiles take it from bf16 high and low
parts, each off by 2^-17).  h as a bf16 high and low part is off by 2^-16, its
sum by 40 u: (2^-16 + 40 u) L.  The bias adds 2 u |y|.  Call the whole d.  An
activation's slope is below 1.13, and its own evaluation (exp2 of an argument t
rounded three times, a reciprocal within 2 u, three products) is off by (12 + 4
|t|) u relative, and by 2^-100 where the exponential leaves the range.  A gated
output multiplies the two: act d_up + |up| d_act + d_act d_up.  Last, bf16: 2^-8."""
import math
import sys

import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
PRECS = [svdq.INT4, svdq.MXFP4]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _matrix(g, rows, K, prec, size):
    """Packed codes (every value of a nibble) and scales, and the values they stand for, in 64 bits."""
    code = torch.randint(0, 16, (rows, K), generator=g, device="cuda", dtype=torch.uint8)
    grp = svdq.group_of(prec)
    if prec == svdq.INT4:
        scale = size * (0.1 + torch.rand(rows, K // grp, generator=g, device="cuda"))
        scale[torch.rand(rows, K // grp, generator=g, device="cuda") < 0.05] = 0.0
        grid, s64 = [0, 1, 2, 3, 4, 5, 6, 7], scale.to(F64)
    else:
        e = torch.randint(-3, 3, (rows, K // grp), generator=g, device="cuda") + int(math.log2(size))
        scale, grid = (e + 127).to(torch.uint8), [0, .5, 1, 1.5, 2, 3, 4, 6]
        s64 = torch.ldexp(torch.ones(rows, K // grp, dtype=F64, device="cuda"), e)
    value = torch.tensor(grid + [-v for v in grid], dtype=F64, device="cuda")[code.int()]
    return code[:, 0::2] + 16 * code[:, 1::2], scale, (value.unflatten(1, (-1, grp)) * s64[..., None]).flatten(1)


def _problem(seed, M, N, K, prec, bias):
    g = torch.Generator(device="cuda").manual_seed(seed)
    xq, xs, X = _matrix(g, M, K, prec, 0.5)
    wq, ws, W = _matrix(g, N, K, prec, 0.25 / math.sqrt(K))
    h = torch.randn(M, 32, generator=g, device="cuda")
    up = (torch.randn(N, 32, generator=g, device="cuda") * 0.1).to(BF)
    b = (torch.randn(N, generator=g, device="cuda") * 0.3).to(BF) if bias else None
    return dict(args=(xq, xs, h, wq, ws, up, b), X=X, W=W, K=K, prec=prec)


def _sums(p, scale_err):
    """Sums in 64 bits, and how far the kernel's may be."""
    _, _, h, _, _, up, b = p["args"]
    y = p["X"] @ p["W"].t().contiguous() + h.to(F64) @ up.to(F64).t().contiguous()
    S, L = p["X"].abs() @ p["W"].abs().t().contiguous(), h.to(F64).abs() @ up.to(F64).abs().t().contiguous()
    if b is not None:
        y = y + b.to(F64)
    return y, ((p["K"] + 8) * U + scale_err) * S + (2.0 ** -16 + 40 * U) * L + 2 * U * y.abs()


def _act(y, d, kind):
    if kind == "gelu":
        t = (2.31 + 0.103 * y * y) * y.abs()
        v = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    else:
        t, v = 1.443 * y.abs(), y * torch.sigmoid(y)
    return v, 1.13 * d + (12 + 4 * t) * U * (v.abs() + 1.13 * d) + 2.0 ** -100


def _close(got, want, d):
    lim = d + 2.0 ** -8 * (want.abs() + d)
    bad = ~((got.to(F64) - want).abs() <= lim)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got.to(F64) - want).abs() - lim).max()))


def _out(M, N):
    """An output between words that no call may touch."""
    buf = torch.full((M * N + 512,), -7.0, dtype=BF, device="cuda")
    return buf, buf[256:256 + M * N].view(M, N)


def _untouched(buf):
    assert bool((buf[:256] == -7).all()) and bool((buf[-256:] == -7).all())


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 48, 64, 65, 130, 256])
@pytest.mark.parametrize("N,K", [(8, 64), (40, 192), (1000, 320), (264, 4096), (16, 11008)])
def test_few_rows(prec, M, N, K):
    _say(f"linear_few prec={prec} {M}x{K}->{N}")
    p = _problem(M, M, N, K, prec, bias=M % 2 == 0)
    y, d = _sums(p, U if prec == svdq.INT4 else 0.0)
    buf, Y = _out(M, N)
    assert svdq.w4a4_linear_few(*p["args"], prec, Y=Y) is Y
    _close(Y, y, d)
    _untouched(buf)
    _close(svdq.w4a4_linear_few(*p["args"], prec, epi=svdq.EPI_GELU_TANH), *_act(y, d, "gelu"))


@pytest.mark.parametrize("K", [32, 96, 160, 224, 288, 1056])
def test_few_rows_odd_blocks(K):
    """MXFP4 rows whose scales start at any byte, and whose last line is not full."""
    for M, N in ((1, 24), (5, 56), (40, 16)):
        p = _problem(K, M, N, K, svdq.MXFP4, True)
        _close(svdq.w4a4_linear_few(*p["args"], svdq.MXFP4), *_sums(p, 0.0))
        p = _problem(K + 1, M, 2 * N, K, svdq.MXFP4, True)
        y, d = _sums(p, 0.0)
        (a, da), u, du = _act(y[:, :N], d[:, :N], "silu"), y[:, N:], d[:, N:]
        _close(svdq.w4a4_linear_gated(*p["args"], svdq.MXFP4), a * u, a.abs() * du + u.abs() * da + da * du)


GATED = [(1, 8, 64), (3, 24, 320), (16, 136, 1024), (17, 200, 192), (64, 72, 512), (65, 8, 64), (100, 136, 320),
         (128, 128, 512), (129, 1000, 256), (300, 264, 768), (513, 392, 96 * 4), (260, 120, 4096), (257, 8, 64), (40, 12296, 320), (200, 7000, 128),
         (64, 28680, 64)]


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("M,F,K", GATED)
@pytest.mark.parametrize("act", [svdq.ACT_SILU, svdq.ACT_GELU_TANH])
def test_gated(prec, M, F, K, act):
    """Few rows and tiles, channels that end inside a tile, K of whole and broken steps."""
    _say(f"linear_gated prec={prec} {M}x{K}->{F} act={act}")
    p = _problem(F, M, 2 * F, K, prec, bias=act == svdq.ACT_SILU)
    y, d = _sums(p, 2.0 ** -15 if prec == svdq.INT4 else 0.0)
    (a, da), u, du = _act(y[:, :F], d[:, :F], "silu" if act == svdq.ACT_SILU else "gelu"), y[:, F:], d[:, F:]
    buf, Y = _out(M, F)
    assert svdq.w4a4_linear_gated(*p["args"], prec, act=act, Y=Y) is Y
    _close(Y, a * u, a.abs() * du + u.abs() * da + da * du)
    _untouched(buf)


@pytest.mark.parametrize("K", [32, 96, 160, 416])
def test_gated_tiles_of_odd_blocks(K):
    p = _problem(K, 300, 2 * 136, K, svdq.MXFP4, True)
    y, d = _sums(p, 0.0)
    (a, da), u, du = _act(y[:, :136], d[:, :136], "silu"), y[:, 136:], d[:, 136:]
    _close(svdq.w4a4_linear_gated(*p["args"], svdq.MXFP4), a * u, a.abs() * du + u.abs() * da + da * du)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("M,F,K", [(1500, 1000, 320), (1029, 2056, 512), (1100, 2000, 4096), (1601, 904, 768),
                                   (1300, 1288, 64), (1500, 1000, 416), (1500, 1000, 96), (2049, 776, 160),
                                   (1025, 1152, 1024), (700, 4104, 256)])
def test_gated_of_many_rows(prec, M, F, K):
    """The tiles: rows and channels that end inside one, K of whole and broken steps, with a bias and without."""
    if prec == svdq.INT4 and K % 64:
        K = 128 * (K // 64)
    _say(f"linear_gated tiles prec={prec} {M}x{K}->{F}")
    p = _problem(F, M, 2 * F, K, prec, bias=M % 2 == 0)
    y, d = _sums(p, 2.0 ** -15 if prec == svdq.INT4 else 0.0)
    buf, Y = _out(M, F)
    for act, name in ((svdq.ACT_SILU, "silu"), (svdq.ACT_GELU_TANH, "gelu")):
        (a, da), u, du = _act(y[:, :F], d[:, :F], name), y[:, F:], d[:, F:]
        svdq.w4a4_linear_gated(*p["args"], prec, act=act, Y=Y)
        _close(Y, a * u, a.abs() * du + u.abs() * da + da * du)
    _untouched(buf)


@pytest.mark.parametrize("prec", PRECS)
def test_gated_of_more_tiles_than_compute_units(prec):
    """Several tiles per block of the persistent kernel, several rounds of the other."""
    M, F, K = 2100, 4488, 256
    p = _problem(1, M, 2 * F, K, prec, True)
    y, d = _sums(p, 2.0 ** -15 if prec == svdq.INT4 else 0.0)
    (a, da), u, du = _act(y[:, :F], d[:, :F], "silu"), y[:, F:], d[:, F:]
    _close(svdq.w4a4_linear_gated(*p["args"], prec), a * u, a.abs() * du + u.abs() * da + da * du)


@pytest.mark.parametrize("prec", PRECS)
def test_large_gates(prec):
    """Gates far out on both sides: act is the gate or nothing, never a NaN."""
    for M in (4, 80):
        p = _problem(9, M, 32, 64, prec, False)
        up = p["args"][5].clone()
        up[:] = 0
        for big in (1e4, 1e30, 3e38):
            h = torch.zeros(M, 32, device="cuda")
            h[:, 0], up[:16, 0], up[16:, 1] = big, 1.0, 1.0
            h[0::2, 0] = -big
            args = p["args"][:2] + (h,) + p["args"][3:5] + (up, None)
            for act in (svdq.ACT_SILU, svdq.ACT_GELU_TANH):
                Y = svdq.w4a4_linear_gated(*args, prec, act=act).float()
                assert not bool(torch.isnan(Y).any()), (M, big, act)
                assert bool((Y[0::2].abs() <= 1e-30).all())


@pytest.mark.parametrize("prec", PRECS)
def test_same_bits_every_time(prec):
    p = _problem(3, 40, 512, 2048, prec, True)
    a = [svdq.w4a4_linear_few(*p["args"], prec) for _ in range(3)]
    b = [svdq.w4a4_linear_gated(*p["args"], prec) for _ in range(3)]
    assert all(torch.equal(a[0], x) for x in a) and all(torch.equal(b[0], x) for x in b)


def test_nothing_to_do():
    p = _problem(3, 4, 32, 64, svdq.INT4, False)
    xq, xs, h, wq, ws, up, _ = p["args"]
    assert svdq.w4a4_linear_few(xq[:0], xs[:0], h[:0], wq, ws, up, None).shape == (0, 32)
    assert svdq.w4a4_linear_gated(xq[:0], xs[:0], h[:0], wq, ws, up, None).shape == (0, 16)
    assert svdq.w4a4_linear_few(xq, xs, h, wq[:0], ws[:0], up[:0], None).shape == (4, 0)
    assert svdq.w4a4_linear_gated(xq, xs, h, wq[:0], ws[:0], up[:0], None).shape == (4, 0)
