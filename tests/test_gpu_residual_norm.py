"""svdq_residual_norm against the formula in 64 bits.

Bound used for the outputs, u = 2^-24 (half a step of fp32).  The sums run over
at most 8 C + 10 <= 74 additions per path (C = 8 chunks of 8 channels per
thread, 6 lane and 4 wave steps), the few other operations add one u each, so
128 u of the magnitudes that enter covers every fp32 error; storing adds half a
step of the output's type (finfo.eps / 2 of the value)."""
import sys

import numpy as np
import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
KINDS = [svdq.NORM_NONE, svdq.NORM_RMS, svdq.NORM_LAYER]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _rand(g, *shape, s=1.0):
    return (torch.randn(*shape, generator=g, dtype=F32) * s).to(BF).cuda()


def _norm64(v, kind, eps):
    """Normalized values, and the magnitude that their fp32 errors scale with."""
    mag = v.abs()
    if kind == svdq.NORM_LAYER:
        mag = mag + v.abs().mean(-1, keepdim=True)
        v = v - v.mean(-1, keepdim=True)
    if kind == svdq.NORM_NONE:
        return v, mag
    rs = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * rs, mag * rs


def _reference(r, y, gate, alpha, post, post_w, pre, pre_w, pre_b, scale, shift, rows, eps):
    """(r', bound of its fp32 error), (x, bound) in 64 bits; rows: modulation row per token, -1 none."""
    D64 = lambda t: t.to(F64)      # noqa: E731
    at, has = rows.clamp_min(0), (rows >= 0)[:, None]
    pick = lambda t, none: torch.where(has, D64(t)[at], torch.full((), none, dtype=F64, device=r.device))  # noqa: E731
    rr, mag = D64(r), D64(r).abs()
    if y is not None:
        t, tm = _norm64(D64(y), post, eps)
        w = D64(post_w) if post_w is not None else 1.0
        g = alpha * (pick(gate, 1.0) if gate is not None else 1.0)
        rr, mag = rr + g * t * w, mag + abs(g * w) * tm
    n, nm = _norm64(rr, pre, eps)
    if pre != svdq.NORM_NONE:
        # an error e of r' changes n by at most 2 e rs (through the value and through the norm and mean)
        v = rr - rr.mean(-1, keepdim=True) if pre == svdq.NORM_LAYER else rr
        rs = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        nm = nm + 2.0 * rs * (mag + mag.mean(-1, keepdim=True))
        nm = nm + n.abs() * (rs * mag.pow(2).mean(-1, keepdim=True).sqrt())
    else:
        nm = mag
    if pre_w is not None:
        n, nm = n * D64(pre_w), nm * D64(pre_w).abs()
    if pre_b is not None:
        n, nm = n + D64(pre_b), nm + D64(pre_b).abs()
    if scale is not None:
        n, nm = n * (1 + pick(scale, 0.0)), nm * (1 + pick(scale, 0.0).abs())
    if shift is not None:
        n, nm = n + pick(shift, 0.0), nm + pick(shift, 0.0).abs()
    return (rr, 128 * U * mag), (n, 128 * U * nm)


def _check(got, ref, bound):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.to(F64) - ref).abs()
    lim = half * (ref.abs() + bound) + bound
    assert bool((err <= lim).all()), f"{int((err > lim).sum())} values off, worst {float((err - lim).max())}"


def _case(M, D, seed, fp32, y=True, gate=True, mod=True, affine=True, B=3):
    g = torch.Generator().manual_seed(seed)
    r = _rand(g, M, D, s=2.0)
    r = (r.float() * 1.0009765625).contiguous() if fp32 else r
    mods = _rand(g, B, 3 * D, s=0.5)
    index = torch.randint(0, B, (M,), generator=g, dtype=torch.int32).cuda()
    return dict(r=r, y=_rand(g, M, D, s=3.0) + 0.5 if y else None, gate=mods[:, 2 * D:] if gate and y else None,
                scale=mods[:, D:2 * D] if mod else None, shift=mods[:, :D] if mod else None,
                post_w=_rand(g, D) if affine and y else None, pre_w=_rand(g, D) if affine else None,
                pre_b=_rand(g, D) if affine else None, mod_index=index)


def _run(c, post, pre, alpha=0.75, eps=1e-6, **kw):
    got_r, got_x = svdq.residual_norm(**c, alpha=alpha, post=post, pre=pre, eps=eps, **kw)
    torch.cuda.synchronize()
    rows = c["mod_index"].long()
    rr, xx = _reference(c["r"], c["y"], c["gate"], alpha, post, c["post_w"], pre, c["pre_w"], c["pre_b"], c["scale"],
                        c["shift"], rows, eps)
    return got_r, got_x, rr, xx


# every width at which the kernel's form changes, and its neighbours
WIDTHS = [8, 16, 504, 512, 520, 1024, 1032, 2040, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(D, fp32):
    for M in (1, 5, 130):
        _say(f"residual_norm M={M} D={D} fp32={fp32}")
        post, pre = KINDS[(D // 8) % 3], KINDS[1 + (D // 8 + M) % 2]
        c = _case(M, D, D + M, fp32)
        got_r, got_x, (r, br), (x, bx) = _run(c, post, pre)
        _check(got_r, r, br)
        _check(got_x, x, bx)


@pytest.mark.parametrize("post", KINDS)
@pytest.mark.parametrize("pre", KINDS)
def test_norms_and_optional_parts(post, pre):
    for k, (gate, mod, affine, fp32) in enumerate([(True, True, True, False), (False, True, False, True),
                                                   (True, False, False, False), (False, False, True, True)]):
        _say(f"residual_norm post={post} pre={pre} gate={gate} mod={mod} affine={affine}")
        c = _case(37, 1544, 10 * post + pre + k, fp32, gate=gate, mod=mod, affine=affine)
        got_r, got_x, (r, br), (x, bx) = _run(c, post, pre)
        _check(got_r, r, br)
        _check(got_x, x, bx)


@pytest.mark.parametrize("fp32", [False, True])
def test_without_block_output_and_without_x(fp32):
    c = _case(9, 640, 5, fp32, y=False)
    got_r, got_x, _, (x, bx) = _run(c, svdq.NORM_NONE, svdq.NORM_LAYER)
    assert got_r is c["r"]
    _check(got_x, x, bx)
    c = _case(9, 640, 6, fp32)
    got_r, got_x, (r, br), _ = _run(c, svdq.NORM_RMS, svdq.NORM_NONE, want_x=False)
    assert got_x is None
    _check(got_r, r, br)


def test_equal_runs_of_rows():
    """Without mod_index the rows are B equal runs; one run is every row."""
    for B, M in ((1, 7), (3, 39)):
        c = _case(M, 264, B, False, B=B)
        c["mod_index"] = torch.arange(M, dtype=torch.int32, device="cuda") // (M // B)
        ref = svdq.residual_norm(**c, pre=svdq.NORM_LAYER)
        c["mod_index"] = None
        got = svdq.residual_norm(**c, pre=svdq.NORM_LAYER)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_rows_outside_the_modulation_take_none():
    c = _case(12, 96, 3, False)
    c["mod_index"][::3] = -1
    c["mod_index"][1::3] = 3
    c["mod_index"][2] = np.iinfo(np.int32).max
    c["mod_index"][5] = np.iinfo(np.int32).min
    got_r, got_x = svdq.residual_norm(**c, pre=svdq.NORM_RMS)
    rows = c["mod_index"].long()
    rows = torch.where((rows >= 0) & (rows < 3), rows, torch.full_like(rows, -1))
    (r, br), (x, bx) = _reference(c["r"], c["y"], c["gate"], 1.0, 0, c["post_w"], 1, c["pre_w"], c["pre_b"],
                                  c["scale"], c["shift"], rows, 1e-6)
    _check(got_r, r, br)
    _check(got_x, x, bx)


@pytest.mark.parametrize("D", [520, 4104])
def test_in_place_and_over_the_block_output(D):
    c = _case(33, D, 8, False)
    ref_r, ref_x = svdq.residual_norm(**c, post=svdq.NORM_RMS, pre=svdq.NORM_LAYER)
    r, y = c["r"].clone(), c["y"].clone()
    c.update(r=r, y=y)
    got_r, got_x = svdq.residual_norm(**c, post=svdq.NORM_RMS, pre=svdq.NORM_LAYER, r_out=r, x=y)
    assert got_r is r and got_x is y
    assert torch.equal(got_r, ref_r) and torch.equal(got_x, ref_x)


@pytest.mark.parametrize("D", [64, 4096])
def test_special_rows(D):
    """Zero rows give the bias and shift (eps > 0); a constant row has no
    LayerNorm part; an infinity or NaN stays in its row."""
    c = _case(8, D, 2, False, affine=False)
    c["r"].zero_()
    c["y"].zero_()
    c["r"][1] = 3.0
    c["r"][3, 5] = float("nan")
    c["y"][5, 7] = float("inf")
    got_r, got_x = svdq.residual_norm(**c, pre=svdq.NORM_LAYER)
    torch.cuda.synchronize()
    want = c["shift"][c["mod_index"].long()]
    for m in (0, 1, 2, 4, 6, 7):
        assert torch.equal(got_x[m], want[m]), m
    assert bool(got_x[3].isnan().all()) and bool(got_x[5].isnan().all())


def test_empty():
    r = torch.empty((0, 64), dtype=BF, device="cuda")
    got_r, got_x = svdq.residual_norm(r, r.clone())
    assert got_r.shape == got_x.shape == (0, 64)


def test_other_stream_and_graph_replays():
    c = _case(50, 2568, 4, True)
    out = dict(r_out=torch.empty_like(c["r"]), x=torch.empty_like(c["y"]))
    call = lambda: svdq.residual_norm(**c, **out, post=svdq.NORM_RMS, pre=svdq.NORM_LAYER)      # noqa: E731
    ref = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = svdq.residual_norm(**c, post=svdq.NORM_RMS, pre=svdq.NORM_LAYER)
    side.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out["r_out"].zero_()
        out["x"].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["r_out"], ref[0]) and torch.equal(out["x"], ref[1])
