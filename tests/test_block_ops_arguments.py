"""What the binding of the calls between the linears does with arguments of a
wrong kind or size.  No GPU."""
import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")


def test_a_plan_that_is_none_is_refused():
    index = torch.zeros(4, dtype=torch.int32)
    for bad in (torch.zeros(4096, dtype=torch.uint8), 7, "plan"):
        with pytest.raises(TypeError, match="LoraPlan"):
            svdq.lora_plan(index, 2, plan=bad)


# Sizes that pass int32, which the C interface takes: their low 32 bits alone
# would be sizes of some other, accepted call.  Meta tensors have no memory.

BIG = 2 ** 32
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
SHAPE, UNSUPPORTED = -2, -4


def m(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


def _refused(status, call, *args, **kw):
    with pytest.raises(svdq.SvdqError) as e:
        call(*args, **kw)
    assert e.value.status == status


@pytest.mark.parametrize("M,D", [(BIG + 8, 8), (8, BIG + 8), (2 ** 31, 8), (2 ** 27, 8)])
def test_residual_norm_of_too_many_values(M, D):
    _refused(SHAPE, svdq.residual_norm, m(M, D))
    _refused(SHAPE, svdq.residual_norm, m(M, D, dtype=F32), m(M, D), want_x=False)


def test_modulation_rows_too_far_apart_or_too_many():
    wide = m(2, BIG + 64)[:, :64]
    _refused(SHAPE, svdq.residual_norm, m(4, 64), m(4, 64), gate=wide)
    _refused(SHAPE, svdq.residual_norm, m(4, 64), scale=m(BIG + 2, 64), mod_index=m(4, dtype=I32))


def test_lora_of_too_many_rows_channels_or_adapters():
    _refused(SHAPE, svdq.lora_plan, m(BIG + 4, dtype=I32), 2)
    _refused(UNSUPPORTED, svdq.lora_plan, m(4, dtype=I32), BIG + 2)
    M, K, N, R, n = 4, 64, 40, 8, 2
    for M, K, N, R in ((M, K, BIG + 40, R), (M, BIG + 64, N, R), (M, K, N, BIG + 8)):
        plan = svdq.LoraPlan(m(4096, dtype=U8), M, n)
        _refused(SHAPE, svdq.lora_linear, m(M, K), m(n, R, K), m(n, N, R), m(n, dtype=F32), plan, m(M, N),
                 work=m(64, dtype=U8))


def test_attention_over_too_many_sequences_or_pages():
    c = svdq.Kv4Cache(1, 16, 1, 64, device="meta")
    for B, width in ((BIG + 2, 1), (2, BIG + 1)):
        _refused(SHAPE, svdq.kv4_attention, m(2, 1, 64), c, m(B, width, dtype=I32), m(B + 1, dtype=I32),
                 m(B, dtype=I32), 1, 16)


def test_bounds_past_int32_are_its_largest_value(monkeypatch):
    """Lengths are int32, so a larger bound is as loose as the largest; a
    negative one stays refused."""
    seen = []

    class Lib:
        def svdq_kv4_attention_workspace_bytes(self, *a):
            seen.append(a[1:])
            return 0
    monkeypatch.setattr(svdq, "lib", lambda: Lib())
    c = svdq.Kv4Cache(1, 16, 1, 64, device="meta")
    svdq.kv4_attention_workspace_bytes(c, 2, 2, 1, BIG + 1, BIG)
    svdq.kv4_attention_workspace_bytes(c, 2, 2, 1, 5 - BIG, -1)
    assert seen == [(2, 2, 1, 2 ** 31 - 1, 2 ** 31 - 1), (2, 2, 1, 0, 0)]
