"""svdq_lora_linear against the formula in 64 bits.

Bound, u = 2^-24: h = X A^T is a sum of K products in fp32 (bf16 products are
exact in it): the matrix instruction adds 32 at a time, so at most K / 32 + 32
+ 3 + slices additions follow one another on any path; (K / 32 + 96) u of
sum |x a| covers them.  h enters the second product as high + low bf16 part,
off by at most 2^-17 |h|: for |h| in [1, 2) the high part leaves at most half
its step, 2^-8; what is left lies in a binade whose step is at most 2^-16, so
the low part leaves at most 2^-17.  The second product has 2 R terms, then base:
(2 R + 4) u of the magnitudes.  Storing adds half a step of bf16 (2^-8 |Y|)."""
import sys

import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _case(M, K, N, R, n, index, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(BF).cuda()      # noqa: E731
    return dict(X=rn(M, K), A=rn(n, R, K, k=K ** -0.5), B=rn(n, N, R), scale=(torch.rand(n, generator=g) + 0.5).cuda(),
                base=rn(M, N)), torch.as_tensor(index, dtype=torch.int32).cuda()


def _check(c, index, Y):
    M, K = c["X"].shape
    n, R, _ = c["A"].shape
    Yd, base = Y.to(F64), c["base"].to(F64)
    for a in sorted(set(index.tolist())):
        rows = torch.nonzero(index == a).flatten()
        if not 0 <= a < n:
            assert torch.equal(Y[rows], c["base"][rows])
            continue
        X, A, B, s = c["X"][rows].to(F64), c["A"][a].to(F64), c["B"][a].to(F64), float(c["scale"][a])
        h, hm = X @ A.t(), X.abs() @ A.abs().t()
        want = base[rows] + s * (h @ B.t())
        eh = (K / 32 + 96) * U * hm + 2.0 ** -17 * h.abs() + 2 * U * h.abs()
        bound = s * (eh @ B.abs().t()) + (2 * R + 4) * U * (s * (h.abs() @ B.abs().t()) + base[rows].abs())
        err = (Yd[rows] - want).abs()
        lim = 2.0 ** -8 * (want.abs() + bound) + bound
        assert bool((err <= lim).all()), (a, int((err > lim).sum()), float((err - lim).max()))


def _run(c, index, **kw):
    plan = svdq.lora_plan(index, c["A"].shape[0])
    Y = svdq.lora_linear(**c, plan=plan, **kw)
    torch.cuda.synchronize()
    return Y


# one token to long runs; widths below, at and above a wave's and a block's; odd multiples of 8
SHAPES = [(1, 8, 8, 8), (1, 4096, 512, 16), (3, 72, 264, 24), (16, 1024, 520, 32), (63, 264, 1000, 40),
          (64, 512, 256, 64), (65, 2048, 328, 72), (130, 264, 2056, 128), (257, 1032, 776, 8), (1000, 328, 1288, 48)]


@pytest.mark.parametrize("M,K,N,R", SHAPES)
@pytest.mark.parametrize("n", [1, 5, 33])
def test_shapes(M, K, N, R, n):
    _say(f"lora M={M} K={K} N={N} R={R} n={n}")
    g = torch.Generator().manual_seed(M + n)
    index = torch.randint(-1, n, (M,), generator=g)
    if M > 100:
        index = index.sort().values if n == 5 else index
    c, index = _case(M, K, N, R, n, index, seed=M)
    _check(c, index, _run(c, index))


@pytest.mark.parametrize("index,n", [([0] * 200, 1), ([-1] * 100, 3), ([2] * 64 + [0] * 65 + [2] * 63, 3),
                                     (list(range(70)), 70), ([5, -7, 2 ** 31 - 1, -2 ** 31, 0, 6], 6),
                                     ([4095, 0, 4095, 7] * 20, 4096)])
def test_assignments(index, n):
    """One adapter for all, none at all, interleaved runs, one row each,
    values outside the range, the most adapters a call takes."""
    _say(f"lora {len(index)} rows, {n} adapters")
    c, idx = _case(len(index), 64, 136, 8, n, index)
    _check(c, idx, _run(c, idx))


def test_in_place_leaves_other_rows_untouched():
    c, idx = _case(90, 256, 320, 16, 4, [i % 5 - 1 for i in range(90)])
    ref = _run(c, idx)
    Y = c["base"].clone()
    c["base"] = Y
    assert _run(c, idx, Y=Y) is Y
    assert torch.equal(Y, ref)


def test_rows_do_not_depend_on_their_neighbours():
    """The same row gives the same bits whatever shares its batch positions."""
    c, idx = _case(300, 768, 264, 32, 6, [(7 * i) % 7 - 1 if i % 3 else i % 6 for i in range(300)])
    ref = _run(c, idx)
    perm = torch.randperm(300, generator=torch.Generator().manual_seed(1)).cuda()
    d = dict(c, X=c["X"][perm].contiguous(), base=c["base"][perm].contiguous())
    assert torch.equal(_run(d, idx[perm].contiguous()), ref[perm])


def test_nan_of_an_unused_adapter_or_row_stays_there():
    c, idx = _case(40, 128, 96, 8, 3, [0, 1] * 20)
    c["A"][2] = float("nan")
    c["B"][2] = float("nan")
    ref = _run(c, idx)
    assert bool(ref.isfinite().all())
    c["X"][7, 3] = float("nan")
    got = _run(c, idx)
    keep = torch.arange(40, device="cuda") != 7
    assert torch.equal(got[keep], ref[keep]) and bool(got[7].isnan().all())


def test_empty():
    c, idx = _case(0, 64, 64, 8, 2, [])
    assert _run(c, idx).shape == (0, 64)
    c, idx = _case(5, 64, 0, 8, 2, [0] * 5)
    assert _run(c, idx).shape == (5, 0)


def test_plan_and_linear_in_a_graph():
    """Plan and linear captured together; new assignments and inputs in the
    same buffers, other work between the replays."""
    c, idx = _case(77, 512, 392, 16, 5, [i % 5 for i in range(77)])
    plan = svdq.lora_plan(idx, 5)
    Y = torch.empty_like(c["base"])
    work = svdq.lora_workspace(77, 512, 16, 5)

    def call():
        svdq.lora_plan(idx, 5, plan=plan)
        svdq.lora_linear(**c, plan=plan, Y=Y, work=work)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        idx.copy_(torch.tensor([(j * (i + 2)) % 6 - 1 for j in range(77)], dtype=torch.int32))
        c["X"].mul_(-1.0)
        Y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _check(c, idx, Y)
        assert torch.equal(Y, _run(c, idx))


def test_two_streams_with_their_own_workspaces():
    c, idx = _case(128, 1024, 512, 32, 8, [i % 9 - 1 for i in range(128)])
    ref = _run(c, idx)
    plan = svdq.lora_plan(idx, 8)
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            out.append(svdq.lora_linear(**c, plan=plan))
    torch.cuda.synchronize()
    for Y in out:
        assert torch.equal(Y, ref)
