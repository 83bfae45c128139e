"""What the binding of the decoding calls does with arguments of a wrong kind or
size where it asks for everything at once, as for device tensors.  No GPU: meta
tensors, which have no memory, say that they lie on device 0, and the library is a
list of the calls that would have reached it."""
import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")

BIG = 2 ** 32
BF, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
SHAPE = -2


class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


class Library:
    def __init__(self):
        self.calls = []

    def svdq_status_string(self, status):
        return b""

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    svdq._tt()
    L = Library()
    monkeypatch.setattr(svdq, "lib", lambda: L)
    monkeypatch.setattr(svdq, "_lib", L)
    monkeypatch.setattr(svdq, "_current_device", lambda: 0)
    monkeypatch.setattr(svdq, "_raw_stream", lambda dev: 0)
    return L


def m(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta").as_subclass(OnDevice)


def _cache(heads=2, dim=64):
    c = svdq.Kv4Cache(4, 16, heads, dim, device="meta")
    c.index = 0
    return c


def _refused(status, L, call, *args, **kw):
    with pytest.raises(svdq.SvdqError) as e:
        call(*args, **kw)
    assert e.value.status == status and not L.calls


def _tree(T=3, B=2, H=4, D=64, width=3, words=1):
    return (m(T, H, D), _cache(dim=D), m(B, width, dtype=I32), m(B + 1, dtype=I32), m(B, dtype=I32), m(T, words, dtype=I32), 4,
            40), dict(out=m(T, H, D), work=m(64, dtype=U8))


def test_calls_of_ordinary_sizes_reach_the_library(library):
    Q, K, cos = m(3, 4, 64), m(3, 2, 64), m(3, 32, dtype=F32)
    svdq.qk_norm_rope(Q, K, cos, cos)
    svdq.kv4_rope_append(_cache(), Q, K, m(3, 2, 64), cos, cos, m(3, dtype=I32))
    args, kw = _tree()
    svdq.kv4_tree_attention(*args, **kw)
    svdq.kv4_tree_plan(_cache(), m(3, dtype=I32), *args[3:5], args[2], 4)
    svdq.kv4_keep_path(_cache(), m(2, 5, dtype=I32), *args[3:5], args[2])
    svdq.rope_table(m(3, 2, dtype=I32), m(32, dtype=F64), m(32, dtype=I32))
    assert [n for n, _ in library.calls] == ["svdq_qk_norm_rope", "svdq_kv4_rope_append", "svdq_kv4_tree_attention",
                                             "svdq_kv4_tree_plan", "svdq_kv4_keep_path", "svdq_rope_table"]


# Sizes that pass int32, which the C interface takes: their low 32 bits alone
# would be sizes of some other, accepted call.

def test_heads_and_tables_too_wide(library):
    cos = m(3, 32, dtype=F32)
    _refused(SHAPE, library, svdq.qk_norm_rope, m(3, 1, BIG + 64), m(3, 1, BIG + 64), cos, cos)
    _refused(SHAPE, library, svdq.qk_norm_rope, m(3, 1, 64), m(3, BIG + 1, 64), cos, cos)
    wide = m(3, BIG + 32, dtype=F32)
    for call, args in ((svdq.qk_norm_rope, ()), (svdq.kv4_rope_append, (_cache(),))):
        more = () if not args else (m(3, 2, 64),)
        last = () if not args else (m(3, dtype=I32),)
        with pytest.raises(ValueError):
            call(*args, m(3, 4, 64), m(3, 2, 64), *more, wide, wide, *last)
    assert not library.calls


def test_masks_too_wide(library):
    args, kw = _tree(words=BIG + 1)
    _refused(SHAPE, library, svdq.kv4_tree_attention, *args, **kw)
    args, kw = _tree(T=0, H=BIG + 4)
    _refused(SHAPE, library, svdq.kv4_tree_attention, *args, **kw)


def test_ranks_too_large(library):
    for call in (svdq.w4a4_linear_few, svdq.w4a4_linear_gated):
        _refused(SHAPE, library, call, m(0, 64, dtype=U8), m(0, 2, dtype=F32), m(0, BIG + 32, dtype=F32), m(0, 64, dtype=U8),
                 m(0, 2, dtype=F32), m(0, BIG + 32), None)


def test_a_negative_bound_on_rows_stays_negative(library, monkeypatch):
    """T of a path: below 0 it is the library's to refuse, however far below."""
    monkeypatch.setattr(svdq, "_launch", lambda *a: 0)
    args, _ = _tree()
    for T in (-1, 6 - BIG):
        svdq.kv4_keep_path(_cache(), m(2, 5, dtype=I32), *args[3:5], args[2], T=T)
        assert library.calls.pop()[1][8] == -1


def test_values_that_are_none_are_refused(library):
    """V is no optional argument: the single checks say so."""
    cos = m(3, 32, dtype=F32)
    with pytest.raises(TypeError, match="V must be a torch tensor"):
        svdq.kv4_rope_append(_cache(), m(3, 4, 64), m(3, 2, 64), None, cos, cos, m(3, dtype=I32))
    assert not library.calls
