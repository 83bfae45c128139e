"""A transformer block as a serving loop runs it: residual + norm + modulation,
4-bit projection, the requests' adapters on top of it, append to the 4-bit
cache, attention over it, projection, residual + norm, MLP, residual.  Every
operator is held against its formula in 64 bits on the values that the chain
feeds it; a decoding step of the whole block is captured and replayed."""
import sys

import numpy as np
import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests import test_gpu_kv4 as kv4
from tests import test_gpu_lora as lora
from tests import test_gpu_residual_norm as norm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
PRECS = [svdq.INT4, svdq.MXFP4]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _ints(*v):
    return torch.tensor(v, dtype=I32, device="cuda")


class Block:
    """Weights of one block, its cache and the buffers of its workspaces."""

    def __init__(self, prec, heads, dim, adapters, pages, page, seed=0):
        self.prec, self.H, self.D, self.C, self.n = prec, heads, dim, heads * dim, adapters
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        C = self.C

        def packed(n, k):
            W = rng.standard_normal((n, k)).astype(np.float32) * k ** -0.5
            bits = (W.view(np.uint32) >> 16).astype(np.uint16)
            absmax = np.full(k, 3.0, np.float32)
            return svdq.to_device(svdq.pack_weights(bits, absmax, prec=prec))
        self.qkv, self.out, self.up, self.down = packed(3 * C, C), packed(C, C), packed(2 * C, C), packed(C, 2 * C)
        rn = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(BF).cuda()      # noqa: E731
        self.A, self.B = rn(adapters, 16, C, k=C ** -0.5), rn(adapters, 3 * C, 16, k=0.1)
        self.s = (torch.rand(adapters, generator=g) + 0.5).cuda()
        self.w1, self.w2, self.b2 = rn(C), rn(C), rn(C, k=0.1)
        self.cache = svdq.Kv4Cache(pages, page, heads, dim, prec)

    def linear(self, x, p, epi=svdq.EPI_NONE):
        return svdq.w4a4_linear(*svdq.quantize_act(x, p["smooth"], p["down"], self.prec), p["wq"], p["wscale"], p["up"],
                                None, self.prec, epi)

    def step(self, r, mods, request, adapter, slots, table, q_start, kv_len, max_q, max_kv):
        """One pass; returns every value that passes between two operators."""
        C, T = self.C, r.shape[0]
        shift1, scale1, gate1, shift2, scale2, gate2 = mods.chunk(6, 1)
        v = {}
        v["x1"] = svdq.residual_norm(r, pre=svdq.NORM_RMS, pre_w=self.w1, scale=scale1, shift=shift1,
                                     mod_index=request)[1]
        v["base"] = self.linear(v["x1"], self.qkv)
        plan = svdq.lora_plan(adapter, self.n)
        v["qkv"] = svdq.lora_linear(v["x1"], self.A, self.B, self.s, plan, v["base"])
        q, k, w = (v["qkv"][:, i * C:(i + 1) * C].view(T, self.H, self.D) for i in range(3))
        svdq.kv4_append(self.cache, k, w, slots)
        v["att"] = svdq.kv4_attention(q, self.cache, table, q_start, kv_len, max_q, max_kv)
        v["y1"] = self.linear(v["att"].view(T, C), self.out)
        v["r1"], v["x2"] = svdq.residual_norm(r, v["y1"], gate=gate1, post=svdq.NORM_RMS, post_w=self.w2,
                                              pre=svdq.NORM_LAYER, pre_w=self.w1, pre_b=self.b2, scale=scale2,
                                              shift=shift2, mod_index=request)
        v["y2"] = self.linear(self.linear(v["x2"], self.up, svdq.EPI_GELU_TANH), self.down)
        v["r2"] = svdq.residual_norm(v["r1"], v["y2"], gate=gate2, pre=svdq.NORM_NONE, mod_index=request, want_x=False)[0]
        return v


def _inputs(seed, T, C, requests):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k)      # noqa: E731
    return rn(T, C, k=2.0).cuda(), rn(requests, 6 * C, k=0.3).to(BF).cuda()


def _verify(b, v, r, mods, request, adapter, table, q_start, lens):
    shift1, scale1, gate1, shift2, scale2, gate2 = mods.chunk(6, 1)
    rows, eps = request.long(), 1e-6
    _, (x, bx) = norm._reference(r, None, None, 1.0, 0, None, svdq.NORM_RMS, b.w1, None, scale1, shift1, rows, eps)
    norm._check(v["x1"], x, bx)
    lora._check(dict(X=v["x1"], A=b.A, B=b.B, scale=b.s, base=v["base"]), adapter, v["qkv"])
    T, P = r.shape[0], b.cache.page_size
    q = v["qkv"][:, :b.C].view(T, b.H, b.D)
    kv = []
    for i, (_, n) in enumerate(lens):
        p = torch.arange(n, device="cuda")
        kv.append(tuple(t.to(F64) for t in svdq.kv4_read(b.cache, (table[i][p // P] * P + p % P).to(I32))))
    starts = q_start.tolist()
    # the new tokens' values are the group quantizer's of what the projection gave
    K, V = (v["qkv"][:, j * b.C:(j + 1) * b.C].reshape(T, b.H, b.D) for j in (1, 2))
    for i, (n, total) in enumerate(lens):
        at = slice(starts[i], starts[i] + n)
        assert torch.equal(kv[i][0][total - n:], kv4._quantized(K[at], b.prec).to(F64))
        assert torch.equal(kv[i][1][total - n:], kv4._quantized(V[at], b.prec).to(F64))
    # that sees the outputs through a buffer with rows behind the last sequence
    out = torch.cat([v["att"], torch.full((1, b.H, b.D), -7.0, dtype=BF, device="cuda")])
    lse = torch.full((T + 1, b.H), 123.0, device="cuda")
    svdq.kv4_attention(q, b.cache, table, q_start, _ints(*[n for _, n in lens]), max(n for n, _ in lens),
                       max(n for _, n in lens), lse=lse[:T])
    x = dict(Q=torch.cat([q, q[:1]]), kv=kv, starts=starts, lens=lens, G=1)
    kv4._verify(x, out, lse, True, 0, b.D ** -0.5)
    (rr, br), (x, bx) = norm._reference(r, v["y1"], gate1, 1.0, svdq.NORM_RMS, b.w2, svdq.NORM_LAYER, b.w1, b.b2,
                                        scale2, shift2, rows, eps)
    norm._check(v["r1"], rr, br)
    norm._check(v["x2"], x, bx)
    (rr, br), _ = norm._reference(v["r1"], v["y2"], gate2, 1.0, 0, None, 0, None, None, None, None, rows, eps)
    norm._check(v["r2"], rr, br)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("heads,dim", [(4, 64), (3, 128)])
def test_prompt_then_chunk_then_tokens(prec, heads, dim):
    """Three requests: their prompts in one ragged pass, a chunk of one beside
    a token of another, then single tokens of all."""
    b = Block(prec, heads, dim, 5, 24, 32, seed=heads)
    table = torch.randperm(24, generator=torch.Generator().manual_seed(3)).to(I32).view(3, 8).cuda()
    have = [0, 0, 0]
    for n, new in enumerate([[90, 33, 1], [1, 70, 0], [1, 1, 1], [1, 1, 1]]):
        print(f"block prec={prec} heads={heads} dim={dim} new={new}", file=sys.stderr, flush=True)
        have = [h + k for h, k in zip(have, new)]
        lens = list(zip(new, have))
        request = torch.cat([torch.full((k,), i, dtype=I32) for i, k in enumerate(new)]).cuda()
        adapter = torch.where(request == 1, -1, 2 * request).to(I32)
        place = torch.cat([torch.arange(h - k, h) for k, h in lens]).cuda()
        slots = (table[request.long(), place // 32] * 32 + place % 32).to(I32)
        q_start = _ints(*np.cumsum([0] + new).tolist())
        r, mods = _inputs(n, len(request), b.C, 3)
        v = b.step(r, mods, request, adapter, slots, table, q_start, _ints(*have), max(new), max(have))
        torch.cuda.synchronize()
        assert all(bool(t.isfinite().all()) for t in v.values())
        _verify(b, v, r, mods, request, adapter, table, q_start, lens)


@pytest.mark.parametrize("prec", PRECS)
def test_decoding_step_in_a_graph(prec):
    """One token of every request through the whole block, captured once; every
    replay, with new inputs, lengths and adapters, equals the eager step."""
    T, H, D, P = 6, 4, 64, 16
    b, e = Block(prec, H, D, 3, 6 * 8, P), Block(prec, H, D, 3, 6 * 8, P)
    table = torch.arange(48, dtype=I32, device="cuda").view(6, 8)
    have = [0, 15, 16, 40, 100, 7]
    for c in (b.cache, e.cache):
        for i, n in enumerate(have):
            p = torch.arange(n, device="cuda")
            K, V = kv4._rand(i, n, H, D), kv4._rand(i + 50, n, H, D)
            svdq.kv4_append(c, K, V, (table[i][p // P] * P + p % P).to(I32))
    request, q_start = torch.arange(T, dtype=I32, device="cuda"), torch.arange(T + 1, dtype=I32, device="cuda")
    r, mods = _inputs(0, T, b.C, T)
    adapter, slots, kv_len = (torch.zeros(T, dtype=I32, device="cuda") for _ in range(3))

    def fill(step):
        for t, s in zip((r, mods), _inputs(step, T, b.C, T)):
            t.copy_(s)
        n = [h + step for h in have]
        adapter.copy_(_ints(*[(i + step) % 4 - 1 for i in range(T)]))
        slots.copy_(_ints(*[int(table[i, k // P]) * P + k % P for i, k in enumerate(n)]))
        kv_len.copy_(_ints(*[k + 1 for k in n]))

    step = lambda x: x.step(r, mods, request, adapter, slots, table, q_start, kv_len, 1, 128)      # noqa: E731
    fill(0)
    step(b)
    want = step(e)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(b)
    for n in range(4):
        fill(n)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step(e)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), (n, k)
        full = [p for i, h in enumerate(have) for p in table[i, :(h + n) // P].tolist()]
        for x, y in ((b.cache.k_codes, e.cache.k_codes), (b.cache.v_codes, e.cache.v_codes)):
            assert torch.equal(x[full], y[full])


@pytest.mark.parametrize("prec", PRECS)
def test_two_batches_on_two_streams(prec):
    """Two batches through blocks of their own at once, one per stream, a long
    prompt beside single tokens: each as alone."""
    H, D, P = 4, 64, 32
    jobs = []
    for n, (new, have) in enumerate([([300, 40], [300, 40]), ([1, 1, 1], [900, 33, 1])]):
        B = len(new)
        table = torch.arange(B * 32, dtype=I32, device="cuda").view(B, 32)
        blocks = [Block(prec, H, D, 3, B * 32, P, seed=n) for _ in range(2)]
        for b in blocks:
            for i, (k, h) in enumerate(zip(new, have)):
                p = torch.arange(h - k, device="cuda")
                svdq.kv4_append(b.cache, kv4._rand(i, h - k, H, D), kv4._rand(i + 9, h - k, H, D),
                                (table[i][p // P] * P + p % P).to(I32))
        request = torch.cat([torch.full((k,), i, dtype=I32) for i, k in enumerate(new)]).cuda()
        place = torch.cat([torch.arange(h - k, h) for k, h in zip(new, have)]).cuda()
        slots = (table[request.long(), place // P] * P + place % P).to(I32)
        r, mods = _inputs(n, len(request), H * D, B)
        args = (r, mods, request, (request % 4 - 1).to(I32), slots, table, _ints(*np.cumsum([0] + new).tolist()),
                _ints(*have), max(new), max(have))
        jobs.append((blocks, args))
    want = [blocks[0].step(*args) for blocks, args in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(jobs[n][0][1].step(*jobs[n][1]))
    for s in streams:
        s.synchronize()
    for n in range(2):
        for v in got[n]:
            for k in want[n]:
                assert torch.equal(v[k], want[n][k]), (n, k)
