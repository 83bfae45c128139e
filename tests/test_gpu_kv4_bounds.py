"""Sequences longer than the caller's bounds: more tiles of rows than blocks
(each takes several in turn), and more keys than the splits were cut for (each
takes a longer part), in the form of few rows and in that of many."""
import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_kv4 import PRECS, _batch, _call, _say, _verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _work(x, max_q, max_kv):
    T, H, _ = x["Q"].shape
    return svdq.kv4_attention_workspace_bytes(x["c"], T, len(x["lens"]), H, max_q, max_kv)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 70)])
@pytest.mark.parametrize("max_q,max_kv", [(20, 200), (20, 3000), (70, 3000), (3, 3000)])
def test_more_rows_than_the_bound(prec, D, causal, window, max_q, max_kv):
    """Two heads per key head: 20 rows make 40, one tile of 128 a sequence (3
    make 6, one of 16), where 150 to 300 rows take three to five (19 to 38)."""
    _say(f"kv4 rows past the bound prec={prec} D={D} causal={causal} window={window} bounds={max_q}, {max_kv}")
    x = _batch(prec, D, 2, 2, 32, [(150, 400), (1, 900), (300, 310), (0, 40), (9, 2500), (211, 211)], seed=21)
    assert (_work(x, max_q, max_kv) > 0) == (max_kv > 200)
    out, lse = _call(x, max_q=max_q, max_kv=max_kv, causal=causal, window=window)
    _verify(x, out, lse, causal, window, D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,max_q", [([(1, 9000), (1, 5000), (1, 1999)], 1), ([(200, 9000), (90, 5000), (1, 64)], 200),
                                        ([(200, 9000), (3, 7001)], 20)])
def test_more_keys_than_the_bound(prec, D, lens, max_q):
    _say(f"kv4 keys past the bound prec={prec} D={D} lens={lens} max_q={max_q}")
    x = _batch(prec, D, 2, 2, 64, lens, seed=22)
    assert _work(x, max_q, 2000) > 0
    out, lse = _call(x, max_q=max_q, max_kv=2000)
    _verify(x, out, lse, True, 0, D ** -0.5)
