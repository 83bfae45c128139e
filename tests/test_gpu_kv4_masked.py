"""What a row does not see cannot reach it: places of the cache that hold the
worst there is, and appended tokens that are not finite."""
import math

import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_kv4 import BF, I32, PRECS, _batch, _cache, _call, _quantized, _rand, _say, _verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,window", [(1, 100), (5, 70), (150, 33), (1, 1)])
def test_pages_before_the_window_may_hold_anything(prec, D, rows, window):
    """A sliding window's caller gives the pages behind it back and points
    their entries at a page that nobody writes (every byte set: NaN scales)."""
    _say(f"kv4 window prec={prec} D={D} rows={rows} window={window}")
    x = _batch(prec, D, 2, 3, 16, [(rows, 500), (1, 30)], seed=rows, pages_extra=1)
    used = set(x["table"][0, :32].tolist()) | set(x["table"][1, :2].tolist())
    spare = next(p for p in range(x["c"].pages) if p not in used)
    first = 500 - rows - window + 1                     # the first key that the first row sees
    x["table"][0, :first // 16] = spare
    out, lse = _call(x, causal=True, window=window)
    _verify(x, out, lse, True, window, D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q", [6, 140])
def test_tokens_that_are_not_finite_stay_in_the_rows_that_see_them(prec, D, q):
    """Infinities and NaN in the last three tokens: the rows before them are
    held against 64 bits over the keys that they see."""
    Hk, G, P, kv = 2, 2, 32, 200
    table = torch.arange(8, dtype=I32, device="cuda").view(1, 8)
    slots = torch.arange(kv, dtype=I32, device="cuda")
    Q = _rand(1, q, Hk * G, D)
    for bad in (math.inf, -math.inf, math.nan):
        K, V = _rand(2, kv, Hk, D), _rand(3, kv, Hk, D)
        K[-3:, :, 5] = bad
        V[-3:, :, 7] = bad
        V[-1] = bad
        c = _cache(8, P, Hk, D, prec)
        svdq.kv4_append(c, K, V, slots)
        k, v = svdq.kv4_read(c, slots)
        assert bool(k.isfinite().all()) and bool(v.isfinite().all())
        lse = torch.empty((q, Hk * G), device="cuda")
        out = svdq.kv4_attention(Q, c, table, torch.tensor([0, q], dtype=I32, device="cuda"),
                                 torch.tensor([kv], dtype=I32, device="cuda"), q, kv, lse=lse)
        x = dict(Q=Q, lens=[(q - 3, kv - 3)], kv=[(k[:-3].double(), v[:-3].double())], starts=[0, q - 3], G=G)
        _verify(x, out[:q - 3], lse[:q - 3], True, 0, D ** -0.5)


def test_the_largest_finite_values():
    """bf16's largest magnitude in K and V: quantized exactly, read finite."""
    for prec in PRECS:
        top = torch.finfo(BF).max
        K = torch.full((4, 1, 64), top, dtype=BF, device="cuda")
        K[1], K[2, :, ::2] = -top, 1.0
        c = _cache(1, 16, 1, 64, prec)
        slots = torch.arange(4, dtype=I32, device="cuda")
        svdq.kv4_append(c, K, K, slots)
        k, v = svdq.kv4_read(c, slots)
        assert torch.equal(k, _quantized(K, prec)) and torch.equal(v, k)


def test_row_bound_far_above_the_rows():
    """max_q as large as the argument allows, many heads per key head."""
    x = _batch(svdq.INT4, 64, 1, 64, 16, [(2, 40), (1, 3)], seed=11)
    out, lse = _call(x, max_q=2 ** 31 - 1, max_kv=2 ** 31 - 4097)
    _verify(x, out, lse, True, 0, 0.125)
    out, lse = _call(x, causal=True, window=2 ** 31 - 1)
    _verify(x, out, lse, True, 0, 0.125)


@pytest.mark.parametrize("prec", PRECS)
def test_calls_on_a_stream_of_their_own(prec):
    """Outputs and workspaces allocated by the call belong to the stream that
    it runs on, whatever the current one."""
    x = _batch(prec, 64, 2, 4, 64, [(1, 4000), (1, 70)], seed=12)
    ref, _ = _call(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        outs = [svdq.kv4_attention(x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"], 1, 4000, stream=stream)
                for _ in range(4)]
        side.synchronize()
        assert all(torch.equal(o[:2], ref[:2]) for o in outs)
