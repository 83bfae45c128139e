"""The 4-bit key / value cache: append and read bit for bit against the group
quantizers in 64 bits, attention against the formula in 64 bits over the values
that the cache holds.

Bound of the attention, u = 2^-24, p the softmax weights, n keys: a score is a
sum of D products in fp32 with at most one more product and sum per group, so
it is off by (D + 8) u scale sum |q k|; the exponent's argument adds 16 u (1 +
|scale score|) (its rounding, the product with log2 e, the hardware's exp2 and
the rescalings).  Call their maximum over the row e: every p is off by e, and
so is their sum.  p enters the second product rounded to bf16: 2^-8.  The sums
over the keys add n u each.  So
  |o - exact| <= (2^-8 + 2 e + 2 n u) sum p |v|  +  2^-8 |o|  (storing).
fp32 and bf16 end at 2^-126: an exponential below it (the largest of a row is
1) may come out as 0 whatever its relative error, and so may its product with
V, which leaves at most 2^-126 max |v| for each of the n keys."""
import math
import sys

import pytest

import w4a4_rank_corrected_quantize_amd as svdq

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


def _rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    x[..., ::17] *= 6.0
    return x.to(BF).cuda()


def _cache(pages, P, H, D, prec):
    """A cache whose unwritten places hold the worst there is: every byte set
    (NaN as fp32 scales, the highest E8M0 byte)."""
    c = svdq.Kv4Cache(pages, P, H, D, prec)
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        t.view(torch.uint8).fill_(255)
    return c


def _quantized(x, prec):
    """The values of the group quantizer, in 64 bits, from its definition."""
    g = svdq.group_of(prec)
    v = x.to(F64).unflatten(-1, (-1, g))
    top = v.abs().amax(-1, keepdim=True)
    if prec == svdq.INT4:
        step = (top / 7).to(F32).to(F64)
        q = torch.where(step > 0, torch.round(v / torch.where(step > 0, step, 1.0)), 0.0)
        return (q * step).to(F32).flatten(-2)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    t = torch.ldexp(v, -e)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device=x.device)
    d = (t.abs().unsqueeze(-1) - grid).abs()
    best = d.amin(-1, keepdim=True)
    near = d == best                                   # one or, at a midpoint, two neighbours
    even = torch.tensor([1, 0] * 4, dtype=torch.bool, device=x.device)
    idx = torch.where(near.sum(-1) > 1, (near & even).int().argmax(-1), near.int().argmax(-1))
    return torch.ldexp(grid[idx] * torch.sign(t), e).to(F32).flatten(-2)


# ------------------------------------------------------------ append and read

@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,P", [(1, 1, 16), (17, 3, 16), (100, 8, 64), (333, 2, 256), (40, 24, 32)])
def test_append_and_read_back(prec, D, T, H, P):
    _say(f"kv4 append prec={prec} D={D} T={T} H={H} P={P}")
    pages = -(-T // P) + 2
    c = _cache(pages, P, H, D, prec)
    K, V = _rand(T, T, H, D), _rand(T + 1, T, H, D)
    K[0] = 0.0
    V[T // 2, 0] = 0.0
    K[T // 2] *= 2.0 ** -120                           # tiny groups: E8M0 near its end, INT4 scales near theirs
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(T))[:T].to(I32).cuda()
    svdq.kv4_append(c, K, V, slots)
    k, v = svdq.kv4_read(c, slots)
    assert torch.equal(k, _quantized(K, prec)) and torch.equal(v, _quantized(V, prec))


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
def test_layout_is_the_documented_one(prec, D):
    """Codes and scales read from the buffers by the layout that svdq.h gives."""
    P, H, T = 32, 2, 50
    c = _cache(3, P, H, D, prec)
    K, V = _rand(1, T, H, D), _rand(2, T, H, D)
    slots = torch.arange(T, dtype=I32, device="cuda") + 20
    svdq.kv4_append(c, K, V, slots)
    k, v = (x.cpu() for x in svdq.kv4_read(c, slots))
    kc, vc, ks, vs = (t.cpu() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales))
    g = svdq.group_of(prec)
    grid = [0, .5, 1, 1.5, 2, 3, 4, 6]

    def value(nib, scale):
        m = float(nib & 7) if prec == svdq.INT4 else grid[nib & 7]
        s = float(scale) if prec == svdq.INT4 else 2.0 ** (int(scale) - 127)
        return float(torch.tensor((-m if nib & 8 else m) * s, dtype=F64).to(F32))
    for t in (0, 11, 12, 43, 44, 49):
        page, place = divmod(int(slots[t]), P)
        run, tok = divmod(place, 16)
        for h in range(H):
            for ch in range(0, D, 3):
                if prec == svdq.MXFP4:
                    b, byte, nib = ch // (D // 4), ch % (D // 4) // 2, ch % 2
                else:
                    gg, b, s, i = ch // 64, ch % 64 // 16, ch % 16 // 8, ch % 8
                    byte, nib = 8 * gg + 4 * s + i % 4, i // 4
                code = int(kc[page, h, run, b, tok, byte]) >> (4 * nib) & 15
                assert value(code, ks[page, h, run, ch // g, tok]) == k[t, h, ch]
                code = int(vc[page, h, run, tok // 4, ch % 16, ch // 32, tok % 4]) >> (4 * (ch % 32 // 16)) & 15
                assert value(code, vs[page, h, run, ch // g, tok]) == v[t, h, ch]


@pytest.mark.parametrize("prec", PRECS)
def test_append_from_a_qkv_product_touches_its_slots_only(prec):
    """K and V as slices of [T][3 H D]; slots outside the cache skip their
    token; every other byte of the cache stays."""
    H, D, T, P = 4, 128, 70, 16
    qkv = _rand(5, T, 3 * H * D)
    K, V = (qkv[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in (1, 2))
    slots = torch.arange(T, dtype=I32, device="cuda") + 13
    slots[3], slots[9], slots[20], slots[21] = -1, 8 * P, 2 ** 31 - 1, -2 ** 31
    c, d = _cache(8, P, H, D, prec), _cache(8, P, H, D, prec)
    svdq.kv4_append(c, K, V, slots)
    keep = (slots >= 0) & (slots < 8 * P)
    svdq.kv4_append(d, K[keep].contiguous(), V[keep].contiguous(), slots[keep].contiguous())
    for x, y in ((c.k_codes, d.k_codes), (c.v_codes, d.v_codes), (c.k_scales, d.k_scales), (c.v_scales, d.v_scales)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    used = torch.zeros(8 * P, dtype=torch.bool, device="cuda")
    used[slots[keep].long()] = True
    free = ~used                                       # [page][place]; place = 16 run + token
    assert bool((c.k_codes.permute(0, 2, 4, 1, 3, 5).reshape(8 * P, -1)[free] == 255).all())
    assert bool((c.v_codes.permute(0, 2, 3, 6, 1, 4, 5).reshape(8 * P, -1)[free] == 255).all())
    k, v = svdq.kv4_read(c, slots)
    want = _quantized(K.contiguous(), prec)
    want[~keep] = 0.0
    assert torch.equal(k, want)


# ------------------------------------------------------------------ attention

def _batch(prec, D, Hk, G, P, lens, seed=0, pages_extra=2):
    """Sequences of (rows, keys) in shuffled pages; block-table entries past a
    sequence's end are invalid."""
    need = [-(-kv // P) for _, kv in lens]
    pages = sum(need) + pages_extra
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(max(need), 1) + 1
    c = _cache(pages, P, Hk, D, prec)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1 if at % 2 else 2 ** 30] * (width - n))
        at += n
    table = torch.tensor(table, dtype=I32, device="cuda")
    starts = [0]
    for q, _ in lens:
        starts.append(starts[-1] + q)
    T = starts[-1] + 3                                  # rows behind the last sequence
    kv_vals = []
    for b, (_, kv) in enumerate(lens):
        K, V = _rand(seed + 10 * b, kv, Hk, D), _rand(seed + 10 * b + 1, kv, Hk, D)
        p = torch.arange(kv, device="cuda")
        slots = (table[b][p // P] * P + p % P).to(I32)
        svdq.kv4_append(c, K, V, slots)
        k, v = svdq.kv4_read(c, slots)
        kv_vals.append((k.to(F64), v.to(F64)))
    Q = _rand(seed + 7, T, Hk * G, D)
    return dict(c=c, Q=Q, table=table, q_start=torch.tensor(starts, dtype=I32, device="cuda"),
                kv_len=torch.tensor([kv for _, kv in lens], dtype=I32, device="cuda"), lens=lens, kv=kv_vals, G=G,
                starts=starts)


def _call(x, max_q=None, max_kv=None, **kw):
    T, H, _ = x["Q"].shape
    lse = torch.full((T, H), 123.0, device="cuda")
    out = torch.full_like(x["Q"], -7.0)
    svdq.kv4_attention(x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"],
                       max_q or max(1, max(q for q, _ in x["lens"])), max_kv or max(1, max(k for _, k in x["lens"])),
                       out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def _verify(x, out, lse, causal, window, scale, dropped=None):
    D = x["Q"].shape[2]
    for b, (q, kv) in enumerate(x["lens"]):
        k, v = x["kv"][b]
        at = x["starts"][b]
        i = torch.arange(q, device="cuda")[:, None] + (kv - q)
        j = torch.arange(kv, device="cuda")[None]
        see = torch.ones((q, kv), dtype=torch.bool, device="cuda")
        if causal:
            see &= j <= i
            if window:
                see &= j > i - window
        if dropped is not None:
            see &= ~dropped[b][None, :kv]
        for h in range(x["Q"].shape[1]):
            Q = x["Q"][at:at + q, h].to(F64)
            kk, vv = k[:, h // x["G"]].contiguous(), v[:, h // x["G"]].contiguous()
            S = (Q @ kk.t().contiguous()) * scale
            mag = (Q.abs() @ kk.abs().t().contiguous()) * scale
            S = S.masked_fill(~see, -math.inf)
            want_lse = torch.logsumexp(S, -1) if kv else torch.full((q,), -math.inf, dtype=F64, device="cuda")
            none = want_lse == -math.inf
            p = torch.where(none[:, None], 0.0, torch.exp(S - torch.where(none, 0.0, want_lse)[:, None]))
            o, pv = p @ vv, p @ vv.abs()
            seen = torch.where(see, mag, 0.0)
            e = ((D + 8) * U * seen + 16 * U * (1 + seen)).amax(-1) if kv else torch.zeros(q, device="cuda")
            n = max(kv, 1)
            lim = (2.0 ** -8 + 2 * e + 2 * n * U)[:, None] * pv
            lim = lim + n * 2.0 ** -126 * (float(vv.abs().max()) if kv else 0.0)
            lim = lim + 2.0 ** -8 * (o.abs() + lim)
            got = out[at:at + q, h].to(F64)
            bad = (got - o).abs() > lim
            assert not bool(bad.any()), (b, h, int(bad.sum()), float(((got - o).abs() - lim).max()))
            gl = lse[at:at + q, h].to(F64)
            assert torch.equal(gl == -math.inf, none)
            dl = (gl - want_lse)[~none].abs() - (2 * e + n * U + 8 * U * (1 + want_lse.abs()))[~none]
            assert not bool((dl > 0).any()), (b, h, float(dl.max()))
    # rows of no sequence
    assert bool((out[x["starts"][-1]:] == -7.0).all()) and bool((lse[x["starts"][-1]:] == 123.0).all())


EDGE = [(1, 1), (1, 15), (1, 16), (1, 17), (0, 40), (1, 63), (1, 64), (1, 65), (1, 0), (1, 129), (1, 300)]
MIXED = [(1, 700), (5, 5), (33, 90), (0, 0), (64, 64), (2, 513), (70, 200), (3, 1), (1, 31)]


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G,P", [(1, 1, 16), (2, 4, 32), (1, 16, 64), (2, 3, 256), (1, 40, 128)])
def test_single_tokens(prec, D, Hk, G, P):
    """The decoding form: one row per sequence, lengths around a page and a
    step, sequences without rows and without keys."""
    _say(f"kv4 attention tokens prec={prec} D={D} Hk={Hk} G={G} P={P}")
    x = _batch(prec, D, Hk, G, P, EDGE, seed=G)
    out, lse = _call(x)
    _verify(x, out, lse, True, 0, D ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50)])
@pytest.mark.parametrize("Hk,G,P", [(2, 1, 16), (1, 8, 64), (3, 2, 128)])
def test_mixed_rows(prec, D, causal, window, Hk, G, P):
    """Chunks of several lengths beside single tokens; rows before the first
    key (more rows than keys) see none under the causal mask."""
    _say(f"kv4 attention mixed prec={prec} D={D} causal={causal} window={window} Hk={Hk} G={G} P={P}")
    x = _batch(prec, D, Hk, G, P, MIXED, seed=G + 3)
    out, lse = _call(x, causal=causal, window=window, scale=0.11)
    _verify(x, out, lse, causal, window, 0.11)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("D", [64, 128])
def test_split_keys(prec, D):
    """Long sequences on few blocks: the keys are split over blocks; short
    ones in the same batch leave splits empty."""
    lens = [(1, 5000), (1, 3), (1, 1), (1, 4097), (1, 0)]
    x = _batch(prec, D, 2, 4, 64, lens, seed=1)
    assert svdq.kv4_attention_workspace_bytes(x["c"], 8, 5, 8, 1, 5000) > 0
    out, lse = _call(x)
    _verify(x, out, lse, True, 0, D ** -0.5)
    lens = [(9, 4000), (20, 600)]
    x = _batch(prec, D, 1, 8, 32, lens, seed=2)
    out, lse = _call(x)
    _verify(x, out, lse, True, 0, D ** -0.5)


@pytest.mark.parametrize("max_q,max_kv", [(1, 1), (1, 100000), (4096, 1), (4096, 100000)])
def test_bounds_do_not_change_what_is_computed(max_q, max_kv):
    """max_q and max_kv far below or above the lengths."""
    x = _batch(svdq.INT4, 64, 2, 2, 32, [(1, 900), (150, 400), (40, 40), (1, 2)], seed=4)
    out, lse = _call(x, max_q=max_q, max_kv=max_kv)
    _verify(x, out, lse, True, 0, 64 ** -0.5)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("rows", [1, 90])
def test_invalid_pages_leave_their_keys_out(prec, rows):
    x = _batch(prec, 128, 1, 2, 16, [(rows, 400), (1, 30)], seed=5)
    dropped = [torch.zeros(400, dtype=torch.bool, device="cuda") for _ in x["lens"]]
    for b, page, bad in ((0, 0, -1), (0, 7, 10 ** 9), (0, 24, -2 ** 31), (1, 0, 2 ** 31 - 1), (1, 1, x["c"].pages)):
        x["table"][b, page] = bad
        dropped[b][16 * page:16 * page + 16] = True
    out, lse = _call(x, causal=False)
    _verify(x, out, lse, False, 0, 128 ** -0.5, dropped)


def test_lengths_past_the_table_are_cut():
    x = _batch(svdq.INT4, 64, 1, 1, 16, [(1, 64), (1, 64)], seed=6)
    x["table"] = x["table"][:, :4].contiguous()
    ref = _call(x)
    x["kv_len"].fill_(2 ** 31 - 1)
    got = _call(x)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    x["kv_len"].fill_(-5)
    got = _call(x)
    assert bool((got[0][:2] == 0).all()) and bool((got[1][:2] == -math.inf).all())


def test_large_scores_and_equal_scores():
    """Scores far apart (one key takes all) and all equal (the mean of V)."""
    x = _batch(svdq.MXFP4, 64, 1, 2, 64, [(3, 300)], seed=8)
    out, lse = _call(x, causal=False, scale=40.0)
    _verify(x, out, lse, False, 0, 40.0)
    x["Q"].zero_()
    out, lse = _call(x, causal=False)
    _verify(x, out, lse, False, 0, 0.125)


def test_nan_row_stays_alone():
    x = _batch(svdq.INT4, 128, 1, 4, 64, [(20, 200)], seed=9)
    ref, _ = _call(x)
    x["Q"][4, 1, 9] = float("nan")
    got, _ = _call(x)
    assert bool(got[4, 1].isnan().all())
    got[4, 1] = ref[4, 1]
    assert torch.equal(got, ref)


def test_strided_queries():
    """Q as a slice of a QKV product."""
    x = _batch(svdq.MXFP4, 64, 2, 2, 32, [(7, 100), (1, 40)], seed=10)
    ref = _call(x)
    T, H, D = x["Q"].shape
    wide = torch.randn(T, 3 * H * D, device="cuda").to(BF)
    wide[:, :H * D] = x["Q"].reshape(T, H * D)
    x["Q"] = wide[:, :H * D].view(T, H, D)
    lse = torch.full((T, H), 123.0, device="cuda")
    out = torch.full((T, H, D), -7.0, dtype=BF, device="cuda")
    svdq.kv4_attention(x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"], 7, 100, out=out, lse=lse)
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("prec", PRECS)
def test_offsets_past_32_bits(prec):
    """A cache whose code buffers are larger than 4 GiB, used at its end."""
    H, D, P, pages = 8, 128, 256, 36000                # 4.7 GB each
    _say("kv4 large cache")
    c = svdq.Kv4Cache(pages, P, H, D, prec)
    assert c.k_codes.numel() > 2 ** 32
    kv = 700
    K, V = _rand(1, kv, H, D), _rand(2, kv, H, D)
    order = [pages - 1, 3, pages - 2]
    table = torch.tensor([order], dtype=I32, device="cuda")
    p = torch.arange(kv, device="cuda")
    slots = (table[0][p // P] * P + p % P).to(I32)
    svdq.kv4_append(c, K, V, slots)
    k, v = svdq.kv4_read(c, slots)
    assert torch.equal(k, _quantized(K, prec)) and torch.equal(v, _quantized(V, prec))
    x = dict(c=c, Q=_rand(3, 4, 16, D), table=table, q_start=torch.tensor([0, 1], dtype=I32, device="cuda"),
             kv_len=torch.tensor([kv], dtype=I32, device="cuda"), lens=[(1, kv)], kv=[(k.to(F64), v.to(F64))], G=2,
             starts=[0, 1])
    out, lse = _call(x)
    _verify(x, out, lse, True, 0, D ** -0.5)


def test_no_rows_and_no_sequences():
    c = _cache(2, 16, 1, 64, svdq.INT4)
    i = lambda *v: torch.tensor(v, dtype=I32, device="cuda")      # noqa: E731
    Q = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    assert svdq.kv4_attention(Q, c, i(0).view(1, 1), i(0, 0), i(0), 1, 1).shape == Q.shape
    Q = torch.zeros((3, 2, 64), dtype=BF, device="cuda")
    out = torch.full_like(Q, 2.0)
    svdq.kv4_attention(Q, c, torch.empty((0, 1), dtype=I32, device="cuda"), i(0), i()[:0], 1, 1, out=out)
    assert bool((out == 2.0).all())
    svdq.kv4_append(c, Q[:0, :1], Q[:0, :1], i()[:0])
    assert svdq.kv4_read(c, i()[:0])[0].shape == (0, 1, 64)


@pytest.mark.parametrize("prec", PRECS)
def test_decoding_steps_in_a_graph(prec):
    """append + attention of one token captured once and replayed as the
    lengths grow: every replay equals the eager calls on a second cache."""
    Hk, G, D, P, B = 2, 4, 128, 16, 3
    kv0 = [600, 15, 31]
    pages = 150
    c, d = _cache(pages, P, Hk, D, prec), _cache(pages, P, Hk, D, prec)
    table = torch.arange(B * 50, dtype=I32, device="cuda").view(B, 50).contiguous()
    for b, kv in enumerate(kv0):
        K, V = _rand(b, kv, Hk, D), _rand(b + 5, kv, Hk, D)
        p = torch.arange(kv, device="cuda")
        for cache in (c, d):
            svdq.kv4_append(cache, K, V, (table[b][p // P] * P + p % P).to(I32))
    q = torch.empty((B, Hk * G, D), dtype=BF, device="cuda")
    k, v = (torch.empty((B, Hk, D), dtype=BF, device="cuda") for _ in range(2))
    slots, kv_len = (torch.zeros(B, dtype=I32, device="cuda") for _ in range(2))
    q_start = torch.arange(B + 1, dtype=I32, device="cuda")
    out = torch.empty_like(q)
    work = svdq.kv4_attention_workspace(c, B, B, Hk * G, 1, 800)

    def fill(step):
        for t, s in ((q, 100), (k, 200), (v, 300)):
            t.copy_(_rand(s + step, *t.shape))
        for b, kv in enumerate(kv0):
            n = kv + step
            slots[b] = int(table[b, n // P]) * P + n % P
            kv_len[b] = n + 1

    def step_on(cache, o, w):
        svdq.kv4_append(cache, k, v, slots)
        svdq.kv4_attention(q, cache, table, q_start, kv_len, 1, 800, out=o, work=w)
    fill(0)
    step_on(c, out, work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_on(c, out, work)
    for step in range(5):
        fill(step)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = torch.empty_like(out)
        step_on(d, ref, None)
        assert torch.equal(out, ref), step


def test_two_streams():
    x = _batch(svdq.MXFP4, 128, 2, 4, 64, [(1, 3000), (1, 2000)], seed=12)
    ref, _ = _call(x)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(svdq.kv4_attention(x["Q"], x["c"], x["table"], x["q_start"], x["kv_len"], 1, 3000))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[:2], ref[:2])
