"""The decoding calls as they are used: a tree of drafted tokens against the same
tokens one at a time, a block's step captured in a graph and replayed as parents,
lengths and paths change on the device, several streams, large offsets, values
that are no numbers."""
import math
import sys

import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_few_gated import _problem
from tests.test_gpu_graph_calls import _replays_match
from tests.test_gpu_kv4 import _batch, _cache, _rand
from tests.test_gpu_rope import _close, _formula, _tables, _weight
from tests.test_gpu_tree import _above, _masks, _parents, _words

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
U = 2.0 ** -24
PRECS = [svdq.INT4, svdq.MXFP4]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _bytes(c):
    return [t.view(U8) for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D,pairs,style", [(64, 32, svdq.ROPE_HALVES), (128, 48, svdq.ROPE_ADJACENT)])
def test_a_tree_is_its_paths(prec, D, pairs, style):
    """Every path of a tree, its tokens one at a time through append and causal attention: the cache holds the same
    bytes where the path is kept, and every node's output is the same but for the roundings of two attentions."""
    _say(f"tree and its paths prec={prec} D={D}")
    H, Hk, P, known, n = 4, 2, 16, 37, 11
    parent = [-1, 0, 0, 1, 3, 2, 5, 4, 7, -1, 9]
    freq, axis = svdq.rope_frequencies([pairs], 10000.0)
    cos, sin = svdq.rope_table(torch.arange(64, dtype=I32, device="cuda").view(64, 1), torch.from_numpy(freq).cuda(),
                               torch.from_numpy(axis).cuda())
    wq, wk = _weight(1, D), _weight(2, D)
    args = dict(style=style, norm_q=wq, norm_k=wk)
    old = [_rand(s, known, h, D) for s, h in ((1, H), (2, Hk), (3, Hk))]
    new = [_rand(s, n, h, D) for s, h in ((4, H), (5, Hk), (6, Hk))]
    table = _i32([[3, 0, 4, 1, 2]])
    q_start = _i32([0, n])

    def start():
        c = _cache(5, P, Hk, D, prec)
        at = torch.arange(known, device="cuda")
        svdq.kv4_rope_append(c, *old, cos, sin, (table[0][at // P] * P + at % P).to(I32), index=at.to(I32), **args)
        return c
    c = start()
    kv_len = _i32([known + n])
    mask, position, slots = svdq.kv4_tree_plan(c, _i32(parent), q_start, kv_len, table, n)
    q = svdq.kv4_rope_append(c, *new, cos, sin, slots, index=position, **args)
    out = svdq.kv4_tree_attention(q, c, table, q_start, kv_len, mask, n, known + n).to(F64)
    snapshot = [t.clone() for t in _bytes(c)]
    for leaf in (8, 6, 10):
        path = []
        while leaf >= 0:
            path.append(leaf)
            leaf = parent[leaf]
        path = path[::-1]
        one = start()
        for i, node in enumerate(path):
            x = [t[node:node + 1] for t in new]
            place = known + i
            assert int(position[node]) == place
            slot = (table[0, place // P] * P + place % P).to(I32).view(1)
            qi = svdq.kv4_rope_append(one, *x, cos, sin, slot, index=_i32([place]), **args)
            assert torch.equal(qi, q[node:node + 1])
            got = svdq.kv4_attention(qi, one, table, _i32([0, 1]), _i32([place + 1]), 1, place + 1).to(F64)
            # both are within (2^-8 + 2^-8) of sums of |p v| <= max |v| (test_gpu_kv4.py): the products' and the
            # stored rounding; the fp32 terms are far below
            lim = 2 * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -14) * float(torch.maximum(old[2].abs().max(), new[2].abs().max()))
            assert float((got[0] - out[node]).abs().max()) <= lim
        # the tree's cache after the move holds the path where the single steps put it
        for t, s in zip(_bytes(c), snapshot):
            t.copy_(s)
        length = svdq.kv4_keep_path(c, _i32([path + [-1]]), q_start, kv_len, table)
        assert length.tolist() == [known + len(path)]
        every = (table[0][torch.arange(known + len(path), device="cuda") // P] * P
                 + torch.arange(known + len(path), device="cuda") % P).to(I32)
        for a, b in zip(svdq.kv4_read(c, every), svdq.kv4_read(one, every)):
            assert torch.equal(a, b)


def _layer(prec, H, Hk, D, F, seed):
    """Packed operands of a block: QKV, output, gated MLP and its second linear (random codes)."""
    M = (H + 2 * Hk) * D, H * D, 2 * F, H * D
    K = H * D, H * D, H * D, F
    L = []
    for i, (n, k) in enumerate(zip(M, K)):
        p = _problem(seed + i, 1, n, k, prec, bias=i == 0)["args"]
        L.append(dict(wq=p[3], ws=p[4], up=p[5], bias=p[6], smooth=torch.rand(k, device="cuda") + 0.5,
                      down=(torch.randn(32, k, device="cuda") * k ** -0.5).to(BF)))
    return L


@pytest.mark.parametrize("prec", PRECS)
def test_step_in_a_graph(prec):
    """A block over two requests' drafted trees: plan, norm, linears of few rows, rotation into the cache, tree
    attention, gated MLP, accepted paths.  Captured once; parents, lengths and paths change on the device between the
    replays, and every replay equals the eager calls on a second cache."""
    _say(f"decoding step in a graph prec={prec}")
    H, Hk, D, F, P, B, most = 4, 2, 64, 320, 16, 2, 12
    torch.manual_seed(3)
    L = _layer(prec, H, Hk, D, F, 40)
    counts = [12, 7]
    T = sum(counts)
    freq, axis = svdq.rope_frequencies([16, 8, 8], 10000.0, svdq.ROPE_AXES_SECTIONS)
    freq, axis = torch.from_numpy(freq).cuda(), torch.from_numpy(axis).cuda()
    q_start = _i32([0, 12, 19])
    table = _i32([[5, 1, 9, 3, 0, 7, 2], [4, 8, 6, 11, 10, 12, 13]])
    parent, path = torch.zeros(T, dtype=I32, device="cuda"), torch.zeros(B, 5, dtype=I32, device="cuda")
    x0 = torch.empty(T, H * D, dtype=BF, device="cuda")
    w1, w2, wk = _weight(1, H * D), _weight(2, H * D), _weight(3, D)

    def linear(x, l, few=True, **kw):
        a = svdq.quantize_act(x, l["smooth"], l["down"], prec)
        f = svdq.w4a4_linear_few if few else svdq.w4a4_linear_gated
        return f(*a, l["wq"], l["ws"], l["up"], l["bias"], prec, **kw)

    def step(c, known, work):
        kv_len = known + (q_start[1:] - q_start[:-1])
        mask, position, slots = svdq.kv4_tree_plan(c, parent, q_start, kv_len, table, most)
        cos, sin = svdq.rope_table(position.view(T, 1).repeat(1, 3), freq, axis)
        _, x = svdq.residual_norm(x0, pre_w=w1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in linear(x, L[0]).split((H * D, Hk * D, Hk * D), 1))
        q = svdq.kv4_rope_append(c, q, k, v, cos, sin, slots, style=svdq.ROPE_HALVES, norm_k=wk)
        att = svdq.kv4_tree_attention(q, c, table, q_start, kv_len, mask, most, 100, work=work)
        r, x = svdq.residual_norm(x0, linear(att.flatten(1), L[1]), pre_w=w2)
        y = linear(linear(x, L[2], few=False, act=svdq.ACT_GELU_TANH), L[3], epi=svdq.EPI_NONE)
        r, _ = svdq.residual_norm(r, y, want_x=False)
        known.copy_(svdq.kv4_keep_path(c, path, q_start, kv_len, table))
        return r

    def fill(i):
        x0.copy_(_rand(70 + i, T, H * D))
        trees = [_parents(10 * i + b, n, 0.6) for b, n in enumerate(counts)]
        parent.copy_(_i32([p for t in trees for p in t]))
        rows = []
        for b, t in enumerate(trees):
            node, up = len(t) - 1, []
            while node >= 0:
                up.append(node)
                node = t[node]
            rows.append((up[::-1][:4] + [-1] * 5)[:5])
        path.copy_(_i32(rows))
    caches, knowns, works = [], [], []
    for _ in range(2):
        c = _cache(14, P, Hk, D, prec)
        at = [(b, i) for b, n in enumerate((30, 45)) for i in range(n)]
        svdq.kv4_append(c, _rand(1, len(at), Hk, D), _rand(2, len(at), Hk, D),
                        _i32([int(table[b, i // P]) * P + i % P for b, i in at]))
        caches.append(c)
        knowns.append(_i32([30, 45]))
        works.append(svdq.kv4_attention_workspace(c, T, B, H, most, 100))
    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                           # what a first call sets up, outside the capture
        step(caches[0], _i32([30, 45]), works[0])
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip(_bytes(caches[0]), _bytes(caches[1])):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step(caches[0], knowns[0], works[0])
    for i in range(4):
        fill(i)
        r.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step(caches[1], knowns[1], None)
        assert torch.equal(r, want), i
        assert torch.equal(knowns[0], knowns[1]) and bool((knowns[0] > _i32([30 + i, 45 + i])).all())
        for a, b in zip(_bytes(caches[0]), _bytes(caches[1])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("prec", PRECS)
def test_single_calls_in_graphs(prec):
    p = _problem(1, 40, 512, 1024, prec, True)["args"]
    Y = torch.empty(40, 512, dtype=BF, device="cuda")
    _replays_match(lambda: svdq.w4a4_linear_few(*p, prec, Y=Y), [Y])
    for M in (3, 300):
        p2 = _problem(2, M, 528, 256, prec, True)["args"]
        Y2 = torch.empty(M, 264, dtype=BF, device="cuda")
        _replays_match(lambda: svdq.w4a4_linear_gated(*p2, prec, Y=Y2), [Y2])
    T = 50
    Q, K, V = _rand(1, T, 4, 64), _rand(2, T, 2, 64), _rand(3, T, 2, 64)
    cos, sin = _tables(4, T, 32)
    Qo, Ko = torch.empty_like(Q), torch.empty_like(K)
    w = _weight(1, 64)
    _replays_match(lambda: svdq.qk_norm_rope(Q, K, cos, sin, norm_q=w, Q_out=Qo, K_out=Ko), [Qo, Ko])
    c = svdq.Kv4Cache(5, 16, 2, 64, prec)
    for t in _bytes(c):
        t.zero_()                                           # the replays start from cleared outputs
    slots = torch.arange(T, dtype=I32, device="cuda") + 7
    _replays_match(lambda: svdq.kv4_rope_append(c, Q, K, V, cos, sin, slots, Q_out=Qo), [Qo, c.k_codes, c.v_codes])


@pytest.mark.parametrize("prec", PRECS)
def test_streams(prec):
    """Calls on two streams at once, and on a stream that is not the current one."""
    p = [_problem(s, 20, 768, 2048, prec, True)["args"] for s in (1, 2)]
    want = [svdq.w4a4_linear_few(*a, prec) for a in p]
    wantg = [svdq.w4a4_linear_gated(*a, prec) for a in p]
    x = _batch(prec, 64, 2, 4, 16, [(9, 300), (30, 31)], seed=5)
    sees = [_above(_parents(b, q, 0.5)) for b, (q, _) in enumerate(x["lens"])]
    m = _masks(x, sees, 1)
    call = lambda **kw: svdq.kv4_tree_attention(x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"], m, 30, 300, **kw)   # noqa: E731
    att = call()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append((svdq.w4a4_linear_few(*p[i % 2], prec), svdq.w4a4_linear_gated(*p[i % 2], prec), call()))
    other = torch.cuda.Stream()
    late = (svdq.w4a4_linear_few(*p[0], prec, stream=other), svdq.w4a4_linear_gated(*p[0], prec, stream=other),
            call(stream=other))
    torch.cuda.synchronize()
    n = x["starts"][-1]
    for i, (a, b, o) in enumerate(got):
        assert torch.equal(a, want[i % 2]) and torch.equal(b, wantg[i % 2]) and torch.equal(o[:n], att[:n])
    assert torch.equal(late[0], want[0]) and torch.equal(late[1], wantg[0]) and torch.equal(late[2][:n], att[:n])


def test_rotation_of_rows_far_apart():
    """Row strides that take offsets past 2^31 elements."""
    big = torch.zeros((1 << 31) + 128, dtype=BF, device="cuda")
    Q = big.as_strided((3, 1, 64), (1 << 30, 64, 1))
    Q.copy_(_rand(1, 3, 1, 64))
    cos, sin = _tables(1, 3, 32)
    q, k = svdq.qk_norm_rope(Q, Q, cos, sin)
    want = _formula(Q, None, cos, sin, torch.arange(3, device="cuda"), svdq.ROPE_ADJACENT, 0)
    _close(q, *want)
    _close(k, *want, key=True)
    svdq.qk_norm_rope(Q, None, cos, sin, Q_out=Q)
    assert torch.equal(Q, q)


@pytest.mark.parametrize("prec", PRECS)
def test_caches_past_32_bits(prec):
    """Slots whose bytes lie past 2^32 in codes and scales."""
    H, D, P = 64, 128, 256
    pages = 6000                                            # 6.3 GB of codes of K alone
    c = svdq.Kv4Cache(pages, P, H, D, prec)
    T, base = 20, (pages - 1) * P + 100
    slots = torch.arange(T, dtype=I32, device="cuda") + base
    Q, K, V = _rand(1, T, 64, D), _rand(2, T, H, D), _rand(3, T, H, D)
    cos, sin = _tables(1, T, 64)
    svdq.kv4_rope_append(c, Q, K, V, cos, sin, slots)
    small = svdq.Kv4Cache(1, P, H, D, prec)
    svdq.kv4_rope_append(small, Q, K, V, cos, sin, slots - (pages - 1) * P)
    for t, s in zip((c.k_codes, c.v_codes, c.k_scales, c.v_scales), (small.k_codes, small.v_codes, small.k_scales, small.v_scales)):
        s[:] = t[-1]
    far, near = _i32([[pages - 1]]), _i32([[0]])
    q_start, kv_len = _i32([0, T]), _i32([100 + T])
    path = _i32([[0, 2, 3, 9, 19]])
    outs = []
    for cache, table in ((c, far), (small, near)):
        mask, _, sl = svdq.kv4_tree_plan(cache, _i32([-1] * T), q_start, kv_len, table, T)
        svdq.kv4_keep_path(cache, path, q_start, kv_len, table)
        outs.append(svdq.kv4_read(cache, sl))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("q", [6, 70])
def test_tokens_that_are_no_numbers_stay_out(prec, q):
    """Drafted tokens with NaN and infinities: rows that do not see them keep their outputs, to the bit."""
    lens = [(q, 300)]
    x = _batch(prec, 64, 2, 4, 16, lens, seed=q)
    see = torch.eye(q, dtype=torch.bool)
    see[:, 0] = True
    m = _masks(x, [see], 3)
    args = (x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"], m, q, 300)
    ref = svdq.kv4_tree_attention(*args)
    bad = torch.full((2, 2, 64), math.nan, dtype=BF, device="cuda")
    bad[1] = math.inf
    at = 300 - q + torch.tensor([2, 4])
    slots = torch.tensor([int(x["table"][0, int(i) // 16]) * 16 + int(i) % 16 for i in at], dtype=I32, device="cuda")
    svdq.kv4_append(x["c"], bad, bad, slots)
    got = svdq.kv4_tree_attention(*args)
    keep = [i for i in range(q) if i not in (2, 4)]
    assert torch.equal(got[keep], ref[keep])
    Q = x["Q"].clone()
    Q[1] = math.nan
    got2 = svdq.kv4_tree_attention(Q, *args[1:])
    rest = [i for i in keep if i != 1]
    assert torch.equal(got2[rest], ref[rest])


@pytest.mark.parametrize("prec", PRECS)
def test_rows_of_linears_stay_apart(prec):
    """A row whose h is no number spoils itself alone; a row's result does not depend on the others."""
    for M in (5, 40, 64, 100):
        p = list(_problem(M, M, 64, 512, prec, True)["args"])
        ref, refg = svdq.w4a4_linear_few(*p, prec), svdq.w4a4_linear_gated(*p, prec)
        p[2] = p[2].clone()
        p[2][3, 7] = math.nan
        got, gotg = svdq.w4a4_linear_few(*p, prec), svdq.w4a4_linear_gated(*p, prec)
        rest = [i for i in range(M) if i != 3]
        assert torch.equal(got[rest], ref[rest]) and torch.equal(gotg[rest], refg[rest])
        assert bool(torch.isnan(got[3]).all()) and bool(torch.isnan(gotg[3]).all())


def test_masks_words_helper():
    see = torch.zeros(2, 40, dtype=torch.bool)
    see[0, 31] = see[1, 32] = True
    assert _words(see, 2).tolist() == [[-2 ** 31, 0], [0, 1]]
