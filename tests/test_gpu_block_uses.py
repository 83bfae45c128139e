"""Ways to use the calls between the linears that a serving loop has and the
other tests do not: lengths and slots advanced on the device inside the captured
step, two captured graphs replayed at once, pages that sequences share."""
import sys

import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_kv4 import BF, F64, I32, PRECS, _cache, _call, _quantized, _rand, _verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


class Decoder:
    """Tokens of B sequences, one a step: the slots come from the table and the
    lengths, the lengths grow, all on the device."""

    def __init__(self, prec, seed, have, D=128, Hk=2, G=4, P=16, width=48):
        B = len(have)
        self.c = _cache(B * width + 1, P, Hk, D, prec)
        order = torch.randperm(B * width, generator=torch.Generator().manual_seed(seed)).to(I32)
        self.table = order.view(B, width).cuda()
        self.kv_len = torch.tensor(have, dtype=I32, device="cuda")
        self.q_start = torch.arange(B + 1, dtype=I32, device="cuda")
        self.rows = torch.arange(B, device="cuda")
        self.P, self.bound = P, width * P
        for b, n in enumerate(have):
            p = torch.arange(n, device="cuda")
            K, V = _rand(seed + b, n, Hk, D), _rand(seed + b + 50, n, Hk, D)
            svdq.kv4_append(self.c, K, V, (self.table[b][p // P] * P + p % P).to(I32))
        self.q = torch.empty((B, Hk * G, D), dtype=BF, device="cuda")
        self.k, self.v = (torch.empty((B, Hk, D), dtype=BF, device="cuda") for _ in range(2))
        self.seed = seed

    def fill(self, n):
        for t, s in ((self.q, 100), (self.k, 200), (self.v, 300)):
            t.copy_(_rand(self.seed + s + n, *t.shape))

    def step(self):
        at = self.kv_len.long()
        slots = (self.table[self.rows, at // self.P] * self.P + at % self.P).to(I32)
        svdq.kv4_append(self.c, self.k, self.v, slots)
        self.kv_len.add_(1)
        return svdq.kv4_attention(self.q, self.c, self.table, self.q_start, self.kv_len, 1, self.bound)


@pytest.mark.parametrize("prec", PRECS)
def test_two_graphs_that_advance_their_own_lengths(prec):
    """Two decoders captured apart and replayed together on two streams, over
    page and step borders: each step equals the eager one of a twin."""
    _say(f"two captured decoders prec={prec}")
    have = ([0, 14, 600, 63], [127, 15, 300])
    run = [Decoder(prec, 10 * i, h) for i, h in enumerate(have)]
    twin = [Decoder(prec, 10 * i, h) for i, h in enumerate(have)]
    graphs, outs = [], []
    for d in run:
        d.fill(0)
        before = d.kv_len.clone()
        d.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(d.step())
        d.kv_len.copy_(before)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in run]
    for n in range(6):
        for d in run + twin:
            d.fill(n)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for d, t, o in zip(run, twin, outs):
            want = t.step()
            torch.cuda.synchronize()
            assert torch.equal(d.kv_len, t.kv_len)
            assert torch.equal(o, want), n


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("rows", [1, 40])
def test_sequences_that_share_pages(prec, rows):
    """A common prompt's pages stand in the tables of all sequences; the pages
    after it are each one's own."""
    Hk, G, D, P, shared = 2, 2, 64, 32, 160
    lens = [(rows, shared + n) for n in (rows, 33 + rows, 200)]
    c = _cache(5 + 3 * 8, P, Hk, D, prec)
    own = torch.arange(24, dtype=I32, device="cuda").view(3, 8) + 5
    table = torch.cat([torch.arange(5, dtype=I32, device="cuda").expand(3, 5), own], 1).contiguous()
    kv = []
    K0, V0 = _rand(1, shared, Hk, D), _rand(2, shared, Hk, D)
    svdq.kv4_append(c, K0, V0, torch.arange(shared, dtype=I32, device="cuda"))
    for b, (_, n) in enumerate(lens):
        K, V = _rand(3 + b, n - shared, Hk, D), _rand(6 + b, n - shared, Hk, D)
        p = torch.arange(shared, n, device="cuda")
        svdq.kv4_append(c, K, V, (table[b][p // P] * P + p % P).to(I32))
        kv.append(tuple(_quantized(torch.cat(t), prec).to(F64) for t in ((K0, K), (V0, V))))
    starts = [0, rows, 2 * rows, 3 * rows]
    x = dict(c=c, Q=_rand(9, 3 * rows + 3, Hk * G, D), table=table, lens=lens, kv=kv, G=G, starts=starts,
             q_start=torch.tensor(starts, dtype=I32, device="cuda"),
             kv_len=torch.tensor([n for _, n in lens], dtype=I32, device="cuda"))
    out, lse = _call(x)
    _verify(x, out, lse, True, 0, D ** -0.5)
