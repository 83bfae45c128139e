"""Channels that do not turn (those behind the pairs of a head that is turned in
part, and tokens without a row in the tables) are passed on as they are, whatever
lies in the channels next to them; turned ones that meet an infinity are what the
formula makes of them."""
import math
import sys

import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_rope import _rand, _tables, _weight

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32
STYLES = [svdq.ROPE_ADJACENT, svdq.ROPE_HALVES]
SIZES = [(64, 8), (64, 16), (128, 24), (128, 32), (256, 40)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _bits(x):
    return x.contiguous().view(torch.int16)


def _heads(D, T=5):
    """Heads with infinities, NaN and both zeros, in turned channels and in others."""
    x = _rand(D, T, 3, D)
    x[0, 0, D - 1], x[0, 1, D - 9], x[0, 2, D // 2 + 3] = math.inf, -math.inf, math.nan
    x[1, 0, 0], x[1, 1, 2], x[1, 2, 5] = math.inf, math.nan, -math.inf
    x[2, 0, 1::2] = -1.0
    x[2, :, 0::2] = -0.0
    x[3, 1] = -0.0
    x[4, 0, 3::8], x[4, 0, D - 5] = math.inf, 3e38
    return x


def _same(got, want):
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(_bits(got)[~nan], _bits(want)[~nan])


@pytest.mark.parametrize("style", STYLES)
@pytest.mark.parametrize("D,pairs", SIZES)
def test_channels_behind_the_pairs(style, D, pairs):
    print(f"behind the pairs style={style} D={D} pairs={pairs}", file=sys.stderr, flush=True)
    x = _heads(D)
    cos, sin = _tables(D, x.shape[0], pairs)
    for got in svdq.qk_norm_rope(x, x, cos, sin, style=style):
        _same(got[..., 2 * pairs:], x[..., 2 * pairs:])
    # with a norm a head with an infinity keeps no finite value but 0, and the infinity itself is no number
    w = _weight(1, D)
    for got in svdq.qk_norm_rope(x, x, cos, sin, style=style, norm_q=w, norm_k=w):
        bad = torch.isinf(x).any(-1)
        behind, was = got[..., 2 * pairs:][bad], x[..., 2 * pairs:][bad]
        assert torch.equal(torch.isnan(behind), torch.isinf(was)) and bool((behind[~torch.isinf(was)] == 0).all())


@pytest.mark.parametrize("style", STYLES)
@pytest.mark.parametrize("D,pairs", SIZES + [(64, 32), (128, 64), (256, 128)])
def test_tokens_without_a_row(style, D, pairs):
    x = _heads(D)
    cos, sin = _tables(D, 4, pairs)
    index = torch.tensor([-1, 4, 2 ** 31 - 1, -2 ** 31, 99], dtype=I32, device="cuda")
    for got in svdq.qk_norm_rope(x, x, cos, sin, style=style, index=index):
        _same(got, x)


@pytest.mark.parametrize("style", STYLES)
def test_turned_channels_meet_as_in_the_formula(style):
    """cos 1 and sin 0 from the tables turn: 0 times an infinity is no number there."""
    D, pairs = 64, 32
    x = _rand(1, 2, 1, D)
    x[0, 0, 4] = math.inf
    cos, sin = torch.ones(2, pairs, device="cuda"), torch.zeros(2, pairs, device="cuda")
    other = 5 if style == svdq.ROPE_ADJACENT else 4 + pairs
    for got in svdq.qk_norm_rope(x, x, cos, sin, style=style):
        want = x.clone()
        want[0, 0, other] = math.nan
        _same(got, want)


@pytest.mark.parametrize("prec", [svdq.INT4, svdq.MXFP4])
@pytest.mark.parametrize("style", STYLES)
@pytest.mark.parametrize("D,pairs", [(64, 16), (128, 24)])
def test_on_into_the_cache(prec, style, D, pairs):
    """Keys that are turned in part, with infinities: the codes of the two calls, and of the channels as they are."""
    x, V = _heads(D), _rand(2, 5, 3, D)
    cos, sin = _tables(D, 3, pairs)
    index = torch.tensor([0, -1, 1, 2, 7], dtype=I32, device="cuda")
    slots = torch.arange(5, dtype=I32, device="cuda") + 3
    caches = [svdq.Kv4Cache(1, 16, 3, D, prec) for _ in range(2)]
    for c in caches:
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            t.view(torch.uint8).zero_()
    q, k = svdq.qk_norm_rope(x, x, cos, sin, style=style, index=index)
    svdq.kv4_append(caches[0], k, V, slots)
    _same(svdq.kv4_rope_append(caches[1], x, x, V, cos, sin, slots, style=style, index=index), q)
    for a, b in zip(*(svdq.kv4_read(c, slots) for c in caches)):
        assert torch.equal(a, b)
    _same(k[1::3], x[1::3])
    _same(q[..., 2 * pairs:], x[..., 2 * pairs:])
