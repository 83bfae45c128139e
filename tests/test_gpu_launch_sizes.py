"""Calls whose plain block counts pass what one launch takes (2^32 - 1 threads
along x)."""
import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_kv4 import I32, PRECS, _batch, _call, _say, _verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


@pytest.mark.parametrize("prec", PRECS)
def test_attention_of_many_sequences_under_a_loose_bound(prec):
    """32768 sequences, all but two without rows, 16 heads, a row bound that
    allows every sequence all rows: 32 tiles x 2^19 would be 2^24 blocks.  The
    first sequence has as many tiles as the bound allows."""
    _say(f"kv4 attention of 32768 sequences prec={prec}")
    x = _batch(prec, 64, 16, 1, 64, [(4000, 4000), (90, 200)], seed=13)
    B, width = 32768, x["table"].shape[1]
    table = torch.full((B, width), -1, dtype=I32, device="cuda")
    table[0], table[-1] = x["table"][0], x["table"][1]
    q_start = torch.full((B + 1,), 4000, dtype=I32, device="cuda")
    q_start[0], q_start[-1] = 0, 4090
    kv_len = torch.zeros(B, dtype=I32, device="cuda")
    kv_len[0], kv_len[-1] = 4000, 200
    x.update(table=table, q_start=q_start, kv_len=kv_len)
    out, lse = _call(x, max_q=2 ** 31 - 1)
    _verify(x, out, lse, True, 0, 64 ** -0.5)


@pytest.mark.parametrize("M", [2 ** 26 + 5, 2 ** 27 - 1])
def test_residual_norm_of_many_short_rows(M):
    """8 channels, four rows per block: 2^24 blocks and more.  Rows do not
    depend on each other, so two calls of half the rows give the same bits."""
    _say(f"residual_norm of {M} rows")
    g = torch.Generator(device="cuda").manual_seed(M)
    r, y = (torch.randn(M, 8, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    got = svdq.residual_norm(r, y, post=svdq.NORM_RMS, pre=svdq.NORM_LAYER)
    half = M // 2
    for rows in (slice(0, half), slice(half, M)):
        want = svdq.residual_norm(r[rows], y[rows], post=svdq.NORM_RMS, pre=svdq.NORM_LAYER)
        assert torch.equal(got[0][rows], want[0]) and torch.equal(got[1][rows], want[1])
