"""Adapters over outputs so wide that a block takes several times 128 channels
in turn: every multiple, widths that end inside one, tiles of few rows, rows
without an adapter (copied and in place)."""
import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_lora import _case, _check, _run, _say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


@pytest.mark.parametrize("M,N,R", [(700, 24584, 8), (700, 33000, 40), (1300, 24008, 72), (4100, 17000, 64), (40, 400008, 16)])
def test_wide_outputs(M, N, R):
    """Runs of 1 to some hundred rows, the last adapter's interleaved with rows
    of none."""
    _say(f"lora wide M={M} N={N} R={R}")
    g = torch.Generator().manual_seed(M)
    index = torch.repeat_interleave(torch.randint(-1, 5, (M,), generator=g), torch.randint(1, M // 6, (M,), generator=g))[:M]
    index[-30::2] = 5
    c, idx = _case(M, 72, N, R, 6, index, seed=N)
    Y = _run(c, idx)
    _check(c, idx, Y)
    c["base"] = base = c["base"].clone()
    assert torch.equal(_run(c, idx, Y=base), Y)
