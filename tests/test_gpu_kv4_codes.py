"""Every rounding decision of the cache's INT4 quantizer that bf16 values can
meet: groups of every mantissa of the largest value, the other values over
every mantissa of the binades below it, at scales from the smallest to the
largest.  Read back bit for bit against the quantizer in 64 bits (on the CPU),
where a quotient of an 8-bit and a 24-bit significand that is no tie lies at
least 2^-33 of its size away from one.  A scale below the smallest normal fp32
is rounded upward, as the formats' definition says."""
import pytest

import w4a4_rank_corrected_quantize_amd as svdq
from tests.test_gpu_kv4 import BF, I32, PRECS, _quantized, _say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    svdq.check_device()


def _exact(x, prec):
    """The values of the group quantizer, by its definition."""
    x = x.cpu()
    if prec == svdq.MXFP4:
        return _quantized(x, prec)
    v = x.double().unflatten(-1, (-1, 64))
    top = v.abs().amax(-1, keepdim=True)
    step = (top / 7).float()
    up = torch.nextafter(step, torch.tensor(torch.inf))
    low = (step < torch.finfo(torch.float32).smallest_normal) & (7 * step.double() < top)
    step = torch.where(low, up, step).double()
    q = torch.where(step > 0, torch.round(v / torch.where(step > 0, step, 1.0)), 0.0)
    return (q * step).float().flatten(-2)


@pytest.mark.parametrize("prec", PRECS)
@pytest.mark.parametrize("exponent", [-126, -125, -110, -98, -97, -96, -20, 0, 1, 60, 126, 127])
def test_every_mantissa(prec, exponent):
    _say(f"kv4 codes prec={prec} 2^{exponent}")
    top = torch.arange(128, 256, dtype=torch.float64) * 2.0 ** (exponent - 7)       # all mantissas of a binade
    rest = torch.cat([torch.arange(128, 256, dtype=torch.float64) * 2.0 ** (exponent - 7 - k) for k in range(6)])
    per = svdq.group_of(prec) - 1
    rest = torch.cat([rest, rest[: -len(rest) % per]]).view(-1, per)
    groups = []
    for t in top:
        v = rest.clamp_max(float(t))                     # the first is the group's largest
        groups.append(torch.cat([t.expand(len(v), 1), v], 1))
    x = torch.cat(groups).to(torch.float32).to(BF)
    x = x * torch.where(torch.rand(x.shape, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0).to(BF)
    x = x.flatten()
    x = torch.cat([x, x[: -x.numel() % 64]]).view(-1, 1, 64).cuda()
    T = x.shape[0]
    c = svdq.Kv4Cache(-(-T // 64), 64, 1, 64, prec)
    slots = torch.arange(T, dtype=I32, device="cuda")
    svdq.kv4_append(c, x, x.flip(0).contiguous(), slots)
    k, v = svdq.kv4_read(c, slots)
    want = _exact(x, prec)
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want.flip(0))
