"""The few-row linears where the row is shorter than the waves of a block would
take: waves that have no part of the product still bring operands of the epilogue.
Calls with other h, up and bias follow each other, beside copies on a second
stream, and each has the bits of its first run, which is within the bound of
tests/test_gpu_few_gated.py."""
import sys

import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_few_gated import U, _act, _close, _problem, _sums

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PRECS = [svdq.INT4, svdq.MXFP4]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("K", [64, 256, 512, 1024])
@pytest.mark.parametrize("M", [17, 40, 64, 200])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_of_less_than_a_part_per_wave(prec, K, M, gated):
    print(f"short rows prec={prec} {M}x{K} gated={gated}", file=sys.stderr, flush=True)
    N = 2 * 520 if gated else 1000
    call = svdq.w4a4_linear_gated if gated else svdq.w4a4_linear_few
    problems = []
    for seed in range(3):
        p = _problem(100 * seed + M, M, N, K, prec, True)
        a = list(p["args"])
        for i in (2, 5, 6):                                     # h, up and bias of another size in every problem
            a[i] = a[i] * 2 ** (2 * seed)
        p["args"] = tuple(a)
        problems.append(p)
    first = []
    for p in problems:
        y, d = _sums(p, U if prec == svdq.INT4 else 0.0)
        got = call(*p["args"], prec)
        if gated:
            F = N // 2
            (v, dv), u, du = _act(y[:, :F], d[:, :F], "silu"), y[:, F:], d[:, F:]
            y, d = v * u, v.abs() * du + u.abs() * dv + dv * du
        _close(got, y, d)
        first.append(got)
    traffic = torch.empty(2, 1 << 26, dtype=torch.uint8, device="cuda")
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        with torch.cuda.stream(other):
            traffic[i % 2].copy_(traffic[1 - i % 2])
        got.append(call(*problems[i % 3]["args"], prec))
    torch.cuda.synchronize()
    assert all(torch.equal(y, first[i % 3]) for i, y in enumerate(got))
