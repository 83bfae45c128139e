"""Attention of trees of up to 1024 drafted tokens, of more drafted tokens than
keys, over pages that are none, and of chains in both attentions.  Bound: that of
tests/test_gpu_kv4.py."""
import math

import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_kv4 import BF, F64, I32, PRECS, U, _batch, _say
from tests.test_gpu_tree import _above, _masks, _parents, _words

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _run(x, masks, call=svdq.kv4_tree_attention, **kw):
    T, H, _ = x["Q"].shape
    out, lse = torch.full((T, H, x["Q"].shape[2]), -7.0, dtype=BF, device="cuda"), torch.full((T, H), 123.0, device="cuda")
    kw = {"max_q": max(q for q, _ in x["lens"]), "max_kv": max(1, max(k for _, k in x["lens"])), **kw}
    args = (x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"]) + (() if masks is None else (masks,))
    call(*args, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert bool((out[x["starts"][-1]:] == -7.0).all()) and bool((lse[x["starts"][-1]:] == 123.0).all())
    return out, lse


def _verify(x, out, lse, sees, scale):
    """sees: [q][kv] bool per sequence."""
    D = x["Q"].shape[2]
    for b, (q, kv) in enumerate(x["lens"]):
        if not q:
            continue
        k, v = x["kv"][b]
        at, see = x["starts"][b], sees[b].cuda()
        for h in range(x["Q"].shape[1]):
            Q = x["Q"][at:at + q, h].to(F64)
            kk, vv = k[:, h // x["G"]].contiguous(), v[:, h // x["G"]].contiguous()
            S = ((Q @ kk.t().contiguous()) * scale).masked_fill(~see, -math.inf)
            mag = (Q.abs() @ kk.abs().t().contiguous()) * scale
            want = torch.logsumexp(S, -1)
            none = ~see.any(-1)
            p = torch.where(none[:, None], 0.0, torch.exp(S - torch.where(none, 0.0, want)[:, None]))
            o, pv = p @ vv, p @ vv.abs()
            seen = torch.where(see, mag, 0.0)
            e = ((D + 8) * U * seen + 16 * U * (1 + seen)).amax(-1)
            lim = (2.0 ** -8 + 2 * e + 2 * kv * U)[:, None] * pv + kv * 2.0 ** -126 * float(vv.abs().max())
            lim = lim + 2.0 ** -8 * (o.abs() + lim)
            bad = ~((out[at:at + q, h].to(F64) - o).abs() <= lim)
            assert not bool(bad.any()), (b, h, int(bad.sum()))
            gl = lse[at:at + q, h].to(F64)
            assert torch.equal(gl == -math.inf, none) and bool((out[at:at + q, h][none] == 0).all())
            dl = ~((gl - want)[~none].abs() <= (2 * e + kv * U + 8 * U * (1 + want.abs()))[~none])
            assert not bool(dl.any()), (b, h)


def _over(q, kv, tree):
    """[q][kv]: the keys before the drafted ones, and of these the tree's."""
    see = torch.ones(q, kv, dtype=torch.bool)
    see[:, max(kv - q, 0):] = tree[:, max(q - kv, 0):]
    return see


LONG = [[(1024, 1500), (1, 700)], [(131, 131), (300, 1000), (513, 3000), (2, 2)], [(256, 4000), (257, 700), (129, 129), (640, 641)]]


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D,Hk,G", [(64, 2, 3), (128, 1, 4), (128, 3, 1)])
@pytest.mark.parametrize("lens", LONG)
def test_long_trees(prec, D, Hk, G, lens):
    """Trees of several tiles of rows, of up to the mask's 1024 tokens."""
    _say(f"long trees prec={prec} D={D} Hk={Hk} G={G} {lens}")
    x = _batch(prec, D, Hk, G, 64, lens, seed=G)
    trees = [_above(_parents(b, q, 0.7)) for b, (q, _) in enumerate(lens)]
    words = -(-max(q for q, _ in lens) // 32)
    out, lse = _run(x, _masks(x, trees, words))
    _verify(x, out, lse, [_over(q, kv, t) for (q, kv), t in zip(lens, trees)], D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D,Hk", [(64, 2), (128, 1), (128, 40)])
def test_more_drafted_tokens_than_keys(prec, D, Hk):
    """The first rows' own places lie before the first key: the others see of them what the mask says."""
    lens = [(9, 4), (40, 1), (70, 69), (33, 2), (5, 300)]
    x = _batch(prec, D, Hk, 4, 16, lens, seed=2)
    trees = [_above(_parents(b, q, 0.8)) for b, (q, _) in enumerate(lens)]
    out, lse = _run(x, _masks(x, trees, 3))
    _verify(x, out, lse, [_over(q, kv, t) for (q, kv), t in zip(lens, trees)], D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("q,Hk", [(5, 2), (60, 2), (60, 40)])
def test_pages_that_are_none(prec, q, Hk):
    """Entries outside the cache, in the prefix and among the drafted tokens: their keys are left out."""
    lens = [(q, 2000), (q + 3, q + 40)]
    x = _batch(prec, 128, Hk, 4, 16, lens, seed=3)
    trees = [_above(_parents(b, n, 0.5)) for b, (n, _) in enumerate(lens)]
    sees = [_over(n, kv, t) for (n, kv), t in zip(lens, trees)]
    for b, page, bad in ((0, 0, -1), (0, 77, 10 ** 9), (0, 124, -2 ** 31), (1, 1, x["c"].pages), (1, (q + 39) // 16, 2 ** 31 - 1)):
        x["table"][b, page] = bad
        sees[b][:, 16 * page:16 * page + 16] = False
    for max_kv in (2000, 100):
        out, lse = _run(x, _masks(x, trees, 2), max_kv=max_kv)
        _verify(x, out, lse, sees, 128 ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,q", [(1, 1), (1, 16), (2, 8), (3, 5), (8, 2), (16, 1)])
@pytest.mark.parametrize("kv", [40, 700, 3000])
def test_a_chain_of_one_tile_has_the_causal_bits(prec, D, G, q, kv):
    """Up to 16 rows both attentions take the same steps of the same tile: the same bits."""
    x = _batch(prec, D, 2, G, 32, [(q, kv)], seed=q)
    chain = _above([i - 1 for i in range(q)])
    out, lse = _run(x, _masks(x, [chain], 1))
    want, wlse = _run(x, None, svdq.kv4_attention)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("q", [7, 40])
def test_queries_out_of_a_wider_product(prec, q):
    """Rows a stride apart, and masks of more words than the rows take."""
    x = _batch(prec, 64, 2, 2, 32, [(q, 300), (q, q)], seed=4)
    trees = [_above(_parents(b, q, 0.5)) for b in range(2)]
    for words in (2, 5):
        want = _run(x, _masks(x, trees, words))
        T, H, D = x["Q"].shape
        wide = torch.full((T, 3 * H * D), 7.0, dtype=BF, device="cuda")
        wide[:, H * D:2 * H * D] = x["Q"].flatten(1)
        got = _run({**x, "Q": wide[:, H * D:2 * H * D].unflatten(1, (H, D))}, _masks(x, trees, words))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert _words(trees[0], 5).shape == (q, 5)
