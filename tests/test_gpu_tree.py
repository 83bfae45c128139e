"""Drafted tokens as a tree: plan and path against walks on the host, attention
against the formula in 64 bits over the values that the cache holds, within the
bound that tests/test_gpu_kv4.py derives for the causal form (the arithmetic is
the same, the mask alone differs)."""
import math
import random
import sys

import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_kv4 import _batch, _cache, _quantized, _rand

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
U = 2.0 ** -24
PRECS = [svdq.INT4, svdq.MXFP4]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _parents(seed, n, chain):
    rng = random.Random(seed)
    return [i - 1 if rng.random() < chain else rng.randint(-1, i - 1) for i in range(n)]


def _above(parent):
    """[n][n] bool: j is i or above it."""
    n = len(parent)
    see = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            see[i, j] = True
            j = parent[j] if parent[j] < j else -1
    return see


def _words(see, words):
    """Masks [n][words] int32 of a [n][m] bool matrix."""
    n, m = see.shape
    bits = torch.zeros(n, 32 * words, dtype=torch.int64)
    bits[:, :min(m, 32 * words)] = see[:, :32 * words].long()
    v = (bits.view(n, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(I32)


# ------------------------------------------------------------------------ plan

@pytest.mark.parametrize("chain", [0.0, 0.6, 1.0])
@pytest.mark.parametrize("counts,P", [((1,), 16), ((8, 0, 31, 32, 33), 32), ((64, 65, 200, 1), 128), ((1024, 3000), 256)])
def test_plan(counts, P, chain):
    _say(f"tree plan {counts} P={P} chain={chain}")
    rng = random.Random(len(counts))
    prefix = [rng.randint(0, 300) for _ in counts]
    parents = [_parents(7 + b, n, chain) for b, n in enumerate(counts)]
    width = max(-(-(p + n) // P) for p, n in zip(prefix, counts)) + 1
    pages = width * len(counts)
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.tensor(order, dtype=I32).view(len(counts), width)
    table[0, 0] = -3                                     # a page that is none
    c = svdq.Kv4Cache(pages, P, 1, 64)
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    T, max_q = starts[-1] + 2, min(max(counts), 1024)
    words = -(-max_q // 32)
    outs = [torch.full((T, words), 77, dtype=I32, device="cuda"), torch.full((T,), 77, dtype=I32, device="cuda"),
            torch.full((T,), 77, dtype=I32, device="cuda")]
    flat = [p for ps in parents for p in ps] + [-1, -1]
    got = svdq.kv4_tree_plan(c, torch.tensor(flat, dtype=I32).cuda(), torch.tensor(starts, dtype=I32).cuda(),
                             torch.tensor([p + n for p, n in zip(prefix, counts)], dtype=I32).cuda(), table.cuda(), max_q,
                             *outs)
    mask, position, slots = (t.cpu() for t in got)
    for b, n in enumerate(counts):
        at = starts[b]
        see = _above(parents[b])
        assert torch.equal(mask[at:at + n], _words(see, words))
        assert position[at:at + n].tolist() == [prefix[b] + int(r.sum()) - 1 for r in see]
        want = [int(table[b, (prefix[b] + i) // P]) for i in range(n)]
        want = [v * P + (prefix[b] + i) % P if v >= 0 else -1 for i, v in enumerate(want)]
        assert slots[at:at + n].tolist() == want
    assert bool((mask[starts[-1]:] == 77).all()) and bool((position[starts[-1]:] == 77).all())
    assert bool((slots[starts[-1]:] == -1).all())


@pytest.mark.parametrize("starts", [(3, 5, 9), (0, 0), (2, 2, 2), (7,)])
def test_rows_of_no_sequence_have_no_slot(starts):
    """A padded step: rows before and behind the sequences write nothing when they are appended with the others."""
    B, T = len(starts) - 1, 300
    c = svdq.Kv4Cache(4, 16, 2, 64)
    table = torch.arange(2 * B, dtype=I32, device="cuda").view(B, 2)
    kv_len = torch.tensor([b - a for a, b in zip(starts, starts[1:])], dtype=I32, device="cuda")
    _, _, slots = svdq.kv4_tree_plan(c, torch.full((T,), -1, dtype=I32, device="cuda"),
                                     torch.tensor(starts, dtype=I32, device="cuda"), kv_len, table, 8,
                                     slots=torch.full((T,), 5, dtype=I32, device="cuda"))
    want = [-1] * T
    for b in range(B):
        for i in range(starts[b], starts[b + 1]):
            want[i] = 32 * b + i - starts[b]
    assert slots.tolist() == want


def test_plan_of_parents_that_are_none():
    """Parents that do not come before their child make it a root; lengths past the table leave no slot."""
    c = svdq.Kv4Cache(4, 16, 1, 64)
    parent = torch.tensor([5, 1, -7, 2 ** 31 - 1, -2 ** 31, 3], dtype=I32, device="cuda")
    q_start = torch.tensor([0, 6], dtype=I32, device="cuda")
    table = torch.tensor([[2]], dtype=I32, device="cuda")
    mask, position, slots = svdq.kv4_tree_plan(c, parent, q_start, torch.tensor([14], dtype=I32, device="cuda"), table, 6)
    assert mask.flatten().tolist() == [1, 2, 4, 8, 16, 32 + 8]
    assert position.tolist() == [8, 8, 8, 8, 8, 9] and slots.tolist() == [40, 41, 42, 43, 44, 45]
    _, _, slots = svdq.kv4_tree_plan(c, parent, q_start, torch.tensor([2], dtype=I32, device="cuda"), table, 6)
    assert slots.tolist() == [-1, -1, -1, -1, 32, 33]
    _, _, slots = svdq.kv4_tree_plan(c, parent, q_start, torch.tensor([400], dtype=I32, device="cuda"), table, 6)
    assert slots.tolist() == [42, 43, 44, 45, 46, 47]        # cut to the table, as the attention cuts it


# ------------------------------------------------------------------- attention

def _call(x, masks, max_q=None, max_kv=None, **kw):
    T, H, _ = x["Q"].shape
    lse = torch.full((T, H), 123.0, device="cuda")
    out = torch.full_like(x["Q"], -7.0)
    svdq.kv4_tree_attention(x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"], masks,
                            max_q or max(1, max(q for q, _ in x["lens"])), max_kv or max(1, max(k for _, k in x["lens"])),
                            out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def _masks(x, sees, words):
    T = x["Q"].shape[0]
    m = torch.full((T, words), -1, dtype=I32)              # rows of no sequence, and bits past a sequence's rows: ones
    for b, (q, _) in enumerate(x["lens"]):
        full = torch.ones(q, 32 * words, dtype=torch.bool)
        full[:, :q] = sees[b][:, :32 * words]
        m[x["starts"][b]:x["starts"][b] + q] = _words(full, words)
    return m.cuda()


def _verify(x, out, lse, sees, words, scale):
    D = x["Q"].shape[2]
    for b, (q, kv) in enumerate(x["lens"]):
        if not q:
            continue
        k, v = x["kv"][b]
        at = x["starts"][b]
        see = torch.ones(q, kv, dtype=torch.bool)
        see[:, kv - q:] = sees[b]
        see[:, kv - q + 32 * words:] = False
        see = see.cuda()
        for h in range(x["Q"].shape[1]):
            Q = x["Q"][at:at + q, h].to(F64)
            kk, vv = k[:, h // x["G"]].contiguous(), v[:, h // x["G"]].contiguous()
            S = ((Q @ kk.t().contiguous()) * scale).masked_fill(~see, -math.inf)
            mag = (Q.abs() @ kk.abs().t().contiguous()) * scale
            want = torch.logsumexp(S, -1)
            none = want == -math.inf
            p = torch.where(none[:, None], 0.0, torch.exp(S - torch.where(none, 0.0, want)[:, None]))
            o, pv = p @ vv, p @ vv.abs()
            seen = torch.where(see, mag, 0.0)
            e = ((D + 8) * U * seen + 16 * U * (1 + seen)).amax(-1)
            lim = (2.0 ** -8 + 2 * e + 2 * kv * U)[:, None] * pv + kv * 2.0 ** -126 * float(vv.abs().max())
            lim = lim + 2.0 ** -8 * (o.abs() + lim)
            bad = (out[at:at + q, h].to(F64) - o).abs() > lim
            assert not bool(bad.any()), (b, h, int(bad.sum()))
            gl = lse[at:at + q, h].to(F64)
            assert torch.equal(gl == -math.inf, none)
            assert bool((out[at:at + q, h][none] == 0).all())
            dl = (gl - want)[~none].abs() - (2 * e + kv * U + 8 * U * (1 + want.abs()))[~none]
            assert not bool((dl > 0).any()), (b, h, float(dl.max()))
    assert bool((out[x["starts"][-1]:] == -7.0).all()) and bool((lse[x["starts"][-1]:] == 123.0).all())


LENS = [(1, 1), (4, 4), (8, 508), (3, 64), (16, 80), (0, 30), (33, 33), (64, 127), (65, 400), (130, 131), (2, 66), (1, 700)]


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G,P", [(1, 1, 16), (2, 4, 64), (1, 8, 256), (3, 3, 32)])
def test_trees(prec, D, Hk, G, P):
    """Trees of 1 to 130 tokens, with prefixes that end anywhere in a step, and without any."""
    _say(f"tree attention prec={prec} D={D} Hk={Hk} G={G} P={P}")
    x = _batch(prec, D, Hk, G, P, LENS, seed=G)
    sees = [_above(_parents(G + b, q, 0.5)) for b, (q, _) in enumerate(LENS)]
    out, lse = _call(x, _masks(x, sees, 5))
    _verify(x, out, lse, sees, 5, D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
def test_any_mask(prec, D):
    """Masks that are no trees: rows that see nothing drafted, or nothing at all; rows past the mask's words."""
    lens = [(7, 7), (12, 300), (70, 90), (40, 40)]
    x = _batch(prec, D, 2, 2, 32, lens, seed=3)
    g = torch.Generator().manual_seed(4)
    sees = [torch.rand(q, q, generator=g) < 0.3 for q, _ in lens]
    for s in sees:
        s[0] = False
        s[-1] = False
    sees[3][:] = False
    for words in (1, 2, 32):
        out, lse = _call(x, _masks(x, sees, words), scale=0.2)
        _verify(x, out, lse, sees, words, 0.2)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D,q", [(64, 3), (128, 4), (64, 40), (128, 64)])
def test_split_keys(prec, D, q):
    """Long prefixes on few blocks: the keys are split; the bounds far off."""
    lens = [(q, 5000), (q, q + 2), (1, 1200)]
    x = _batch(prec, D, 1, 4, 64, lens, seed=q)
    sees = [_above(_parents(b, n, 0.7)) for b, (n, _) in enumerate(lens)]
    m = _masks(x, sees, 2)
    out, lse = _call(x, m)
    _verify(x, out, lse, sees, 2, D ** -0.5)
    for mq, mk in ((1, 100000), (4096, 1)):
        out, lse = _call(x, m, max_q=mq, max_kv=mk)
        _verify(x, out, lse, sees, 2, D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D,Hk", [(64, 8), (128, 4)])
@pytest.mark.parametrize("long", [0, 1, 5])
def test_many_rows(prec, D, Hk, long):
    """Enough trees for tiles of 128 rows and of 64, with the keys whole (no prefix above 150) or divided evenly over the
    blocks (1500 and 7500), for trees of every remainder of a tile."""
    _say(f"many rows prec={prec} D={D} Hk={Hk} long={long}")
    rng = random.Random(D + long)
    counts = [40, 33, 16, 48, 64, 20, 5, 0, 47, 32, 31, 63, 1, 44, 39, 55]
    lens = [(q, q + (rng.randint(0, 150) if not long else rng.choice([0, 30, 1500 * long // (1 + b % 3)])))
            for b, q in enumerate(counts)]
    x = _batch(prec, D, Hk, 4, 64, lens, seed=D)
    sees = [_above(_parents(b, n, 0.7)) for b, (n, _) in enumerate(lens)]
    out, lse = _call(x, _masks(x, sees, 2))
    _verify(x, out, lse, sees, 2, D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D,Hk", [(64, 3), (128, 1)])
@pytest.mark.parametrize("B", [64, 65, 150])
def test_many_sequences(prec, D, Hk, B):
    """As many trees as the division looks at at once, and more; some without rows, some without a prefix."""
    _say(f"many sequences prec={prec} D={D} Hk={Hk} B={B}")
    rng = random.Random(B + D)
    lens = [(q, q + rng.choice([0, 40, 130, 700])) for q in (rng.choice([0, 3, 12, 18, 33, 40]) for _ in range(B))]
    lens[0], lens[-1] = (40, 740), (0, 0)
    x = _batch(prec, D, Hk, 8, 32, lens, seed=B)
    sees = [_above(_parents(b, n, 0.6)) for b, (n, _) in enumerate(lens)]
    out, lse = _call(x, _masks(x, sees, 2))
    _verify(x, out, lse, sees, 2, D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D,Hk", [(64, 8), (128, 4)])
def test_divided_keys_captured_and_on_two_streams(prec, D, Hk):
    """The even division follows the lengths that a replay finds, reads nothing of a workspace that it has not written,
    and two calls at once keep apart."""
    _say(f"divided keys captured prec={prec} D={D} Hk={Hk}")
    counts = [40, 33, 16, 48, 64, 20, 5, 0, 47, 32, 31, 63, 1, 44, 39, 55]
    x, y = (_batch(prec, D, Hk, 4, 64, [(q, q + (b * (211 + 89 * k)) % 1700) for b, q in enumerate(counts)], seed=D + k)
            for k in range(2))
    masks = [_masks(z, [_above(_parents(b, n, 0.5)) for b, n in enumerate(counts)], 2) for z in (x, y)]
    T, H = x["Q"].shape[:2]
    work = [svdq.kv4_attention_workspace(z["c"], T, 16, H, 64, 1800) for z in (x, y)]
    assert all(w is not None for w in work)
    out, lse = [torch.empty_like(z["Q"]) for z in (x, y)], [torch.empty(T, H, device="cuda") for _ in range(2)]

    def call(k, **kw):
        z = (x, y)[k]
        return svdq.kv4_tree_attention(z["Q"], z["c"], z["table"], z["q_start"], z["kv_len"], masks[k], 64, 1800,
                                       out=out[k], lse=lse[k], work=work[k], **kw)

    def clear(k):
        out[k].fill_(-7.0), lse[k].fill_(123.0), work[k].fill_(255)

    full = x["kv_len"].clone()
    lengths = [full, torch.minimum(full, x["q_start"].diff() + 300), x["q_start"].diff(), torch.minimum(full, torch.full_like(full, 900))]
    want = []
    for n in lengths:
        x["kv_len"].copy_(n)
        clear(0), call(0)
        want.append((out[0].clone(), lse[0].clone()))
    assert all(bool(torch.isfinite(o.float()).all()) for o, _ in want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(0)
    for i in (1, 0, 3, 2, 1):
        x["kv_len"].copy_(lengths[i])
        clear(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i][0]) and torch.equal(lse[0], want[i][1]), i
    x["kv_len"].copy_(full)
    clear(1), call(1)
    other = out[1].clone(), lse[1].clone()
    clear(0), clear(1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for k, st in enumerate(streams):
            call(k, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0][0]) and torch.equal(lse[0], want[0][1])
    assert torch.equal(out[1], other[0]) and torch.equal(lse[1], other[1])


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
def test_a_chain_is_the_causal_form(prec, D):
    """A chain's rows see what the causal mask lets them see: the same bits."""
    lens = [(1, 40), (9, 300), (30, 30), (100, 1000)]
    x = _batch(prec, D, 2, 4, 16, lens, seed=6)
    sees = [_above([i - 1 for i in range(q)]) for q, _ in lens]
    out, lse = _call(x, _masks(x, sees, 4))
    want, wlse = torch.full_like(out, -7.0), torch.full_like(lse, 123.0)
    svdq.kv4_attention(x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"], 100, 1000, out=want, lse=wlse)
    _verify(x, out, lse, sees, 4, D ** -0.5)
    _verify(x, want, wlse, sees, 4, D ** -0.5)


# ------------------------------------------------------------------------ path

@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D,H,P", [(64, 3, 16), (128, 2, 64), (128, 1, 256)])
def test_keep_path(prec, D, H, P):
    """Kept tokens hold what they held, at their new places; every other byte of the cache stays."""
    _say(f"keep path prec={prec} D={D} H={H} P={P}")
    counts = [8, 1, 100, 40, 0, 64, 5]
    prefix = [0, 17, 250, 31, 9, 64, 100]
    paths = [[0, 3, 4, 7], [0], list(range(1, 100, 2)), [], [], list(range(64)), [4]]
    rng = random.Random(D)
    width = max(-(-(p + n) // P) for p, n in zip(prefix, counts))
    pages = width * len(counts)
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.tensor(order, dtype=I32).view(len(counts), width)
    c = _cache(pages, P, H, D, prec)
    total = pages * P
    K, V = _rand(1, total, H, D), _rand(2, total, H, D)
    every = torch.arange(total, dtype=I32, device="cuda")
    svdq.kv4_append(c, K, V, every)
    wantk, wantv = svdq.kv4_read(c, every)
    slot = lambda b, place: int(table[b, place // P]) * P + place % P       # noqa: E731
    newk, newv = wantk.clone(), wantv.clone()
    for b, path in enumerate(paths):
        for i, node in enumerate(path):
            newk[slot(b, prefix[b] + i)] = wantk[slot(b, prefix[b] + node)]
            newv[slot(b, prefix[b] + i)] = wantv[slot(b, prefix[b] + node)]
    longest = max(len(p) for p in paths) + 1
    dirt = [[-1, 5, 3], [0, 0, 1], [99, 99, 2], [-1], [0, 1], [63, 1], [4]]   # what follows a path's end
    rows = [(p + dirt[b] + [-1] * longest)[:longest] for b, p in enumerate(paths)]
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    got = svdq.kv4_keep_path(c, torch.tensor(rows, dtype=I32).cuda(), torch.tensor(starts, dtype=I32).cuda(),
                             torch.tensor([p + n for p, n in zip(prefix, counts)], dtype=I32).cuda(), table.cuda())
    assert got.tolist() == [p + len(q) for p, q in zip(prefix, paths)]
    k, v = svdq.kv4_read(c, every)
    assert torch.equal(k, newk) and torch.equal(v, newv)


def test_keep_path_leaves_bad_pages_out():
    c = _cache(4, 16, 1, 64, svdq.MXFP4)
    every = torch.arange(64, dtype=I32, device="cuda")
    svdq.kv4_append(c, _rand(1, 64, 1, 64), _rand(2, 64, 1, 64), every)
    k0, v0 = svdq.kv4_read(c, every)
    table = torch.tensor([[1, 7]], dtype=I32, device="cuda")                 # places 16 .. have no page
    path = torch.tensor([[1, 4, 6, -1]], dtype=I32, device="cuda")           # places 13, 16 (none), 18 (none)
    n = svdq.kv4_keep_path(c, path, torch.tensor([0, 8], dtype=I32, device="cuda"),
                           torch.tensor([20], dtype=I32, device="cuda"), table)
    k, v = svdq.kv4_read(c, every)
    k0[16 + 12], v0[16 + 12] = k0[16 + 13].clone(), v0[16 + 13].clone()
    assert n.tolist() == [15] and torch.equal(k, k0) and torch.equal(v, v0)
