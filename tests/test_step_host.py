"""The operators around the selection on the host: the C entry points refuse
what they cannot do before any CUDA call, the binding refuses what the C
entry points cannot see, and the rotary frequencies are their formulas."""

import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_fp32_gb300 as tk  # noqa: E402
from sparse_attention_indexer_fp32_gb300 import _step  # noqa: E402
from sparse_attention_indexer_fp32_gb300 import build as cuda_build  # noqa: E402

SOME = 0x1000


@pytest.fixture(scope="module")
def lib():
    if cuda_build.is_stale():
        cuda_build.build()
    return tk.load_library()


def _status(lib, name, kind, base, **changes):
    a = kind(**{**base, **changes})
    fn = getattr(lib, name)
    fn.argtypes, fn.restype = [ctypes.POINTER(kind), ctypes.c_void_p], ctypes.c_int
    return fn(ctypes.byref(a), None)


ROTARY = dict(x=SOME, x_token_stride=128, x_head_stride=64, out=SOME, out_token_stride=128, out_head_stride=64,
              positions=SOME, frequencies=SOME, T=2, H=2, D=64, rotated=64, offset=0, layout=0, type=0, scale=1.0)


def test_rotary_refusals(lib):
    bad = [dict(T=-1), dict(H=-1), dict(D=0), dict(D=1026, rotated=64), dict(rotated=0), dict(rotated=33),
           dict(rotated=66), dict(offset=2), dict(offset=-2, rotated=32), dict(type=3), dict(type=-1), dict(layout=2),
           dict(scale=math.inf), dict(scale=math.nan), dict(x=None), dict(out=None), dict(positions=None),
           dict(frequencies=None), dict(x=SOME + 1), dict(out=SOME + 1), dict(positions=SOME + 2),
           dict(positions=SOME + 4, positions_64=1), dict(frequencies=SOME + 4), dict(slots=SOME + 2, num_pages=1, page_size=1),
           dict(slots=SOME, num_pages=-1, page_size=1), dict(slots=SOME, num_pages=1, page_size=-1),
           dict(slots=SOME, num_pages=2 ** 62, page_size=64)]
    for change in bad:
        assert _status(lib, "sparse_rotary", _step._RotaryArgs, ROTARY, **change) == tk.Status.EINVAL, change
    for change in (dict(T=0), dict(H=0), dict(slots=SOME, num_pages=0, page_size=4)):
        assert _status(lib, "sparse_rotary", _step._RotaryArgs, ROTARY, **change) == tk.Status.OK, change
    assert lib.sparse_rotary(None, None) == tk.Status.EINVAL


SCORES = dict(q=SOME, q_seq_stride=128, q_token_stride=128, q_head_stride=64, weights=SOME, keys=SOME,
              key_page_stride=1024, key_token_stride=64, lengths=SOME, page_table=SOME, table_stride=4, table_width=4,
              out=SOME, out_seq_stride=64, out_token_stride=64, num_pages=8, width=64, page_size=16, B=2, T=1, H=2,
              D=64, type=0)


def test_scores_refusals(lib):
    bad = [dict(type=2), dict(type=4), dict(B=-1), dict(T=-1), dict(H=0), dict(H=129), dict(D=0), dict(D=136),
           dict(D=60), dict(D=72, type=3), dict(width=-1), dict(width=2 ** 31), dict(width=65), dict(page_size=0),
           dict(page_size=-1), dict(table_stride=-1), dict(num_pages=-1), dict(q=None), dict(weights=None),
           dict(keys=None), dict(lengths=None), dict(page_table=None), dict(out=None), dict(keys=SOME + 8),
           dict(key_page_stride=1028), dict(key_token_stride=68), dict(q=SOME + 1), dict(weights=SOME + 2),
           dict(key_scales=SOME + 2), dict(lengths=SOME + 2), dict(page_table=SOME + 2), dict(out=SOME + 2)]
    for change in bad:
        assert _status(lib, "sparse_indexer_scores", _step._ScoresArgs, SCORES, **change) == tk.Status.EINVAL, change
    for change in (dict(B=0), dict(T=0), dict(width=0)):
        assert _status(lib, "sparse_indexer_scores", _step._ScoresArgs, SCORES, **change) == tk.Status.OK, change
    assert lib.sparse_indexer_scores(None, None) == tk.Status.EINVAL


ATTENTION = dict(q=SOME, q_seq_stride=256, q_token_stride=256, q_head_stride=64, k=SOME, k_page_stride=2048,
                 k_token_stride=128, k_head_stride=64, v=SOME, v_page_stride=2048, v_token_stride=128,
                 v_head_stride=64, indices=SOME, page_table=SOME, table_stride=4, table_width=4, out=SOME,
                 num_pages=8, page_size=16, B=2, T=1, Hq=4, Hkv=2, D=64, Dv=64, K=8, type=0, scale=0.125)


def test_attention_refusals(lib):
    bad = [dict(type=2), dict(type=3), dict(B=-1), dict(T=-1), dict(Hkv=0), dict(Hq=3), dict(Hq=-2), dict(K=-1),
           dict(D=0), dict(D=60), dict(D=264), dict(Dv=0), dict(Dv=4), dict(Dv=264), dict(scale=math.nan),
           dict(scale=math.inf), dict(softcap=-1.0), dict(softcap=math.nan), dict(softcap=math.inf), dict(num_pages=-1),
           dict(page_size=-1), dict(table_width=-1), dict(table_stride=-1), dict(slopes=SOME),
           dict(page_table=None, first=SOME), dict(page_table=None, query_positions=SOME), dict(q=None), dict(k=None),
           dict(v=None), dict(indices=None), dict(out=None), dict(k=SOME + 8), dict(v=SOME + 8), dict(out=SOME + 8),
           dict(q=SOME + 1), dict(k_page_stride=2052), dict(k_token_stride=132), dict(k_head_stride=68),
           dict(v_page_stride=2052), dict(v_token_stride=132), dict(v_head_stride=68), dict(indices=SOME + 2),
           dict(page_table=SOME + 2), dict(query_positions=SOME + 2), dict(first=SOME + 2), dict(lse=SOME + 2),
           dict(slopes=SOME + 2, query_positions=SOME), dict(num_pages=2 ** 60)]
    for change in bad:
        assert _status(lib, "sparse_attention", _step._AttentionArgs, ATTENTION, **change) == tk.Status.EINVAL, change
    for change in (dict(B=0), dict(T=0), dict(Hq=0)):
        assert _status(lib, "sparse_attention", _step._AttentionArgs, ATTENTION, **change) == tk.Status.OK, change
    assert lib.sparse_attention(None, None) == tk.Status.EINVAL


def test_binding_refuses_tensors_off_the_gpu():
    """There is no CPU path: host tensors are refused by name."""
    x = torch.zeros((2, 2, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        tk.rotary(x, torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))
    q = torch.zeros((1, 1, 2, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        tk.indexer_scores(q, torch.zeros((1, 1, 2)), q[0], torch.zeros((1, 1), dtype=torch.int32),
                          torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        tk.sparse_attention(q, q, q, torch.zeros((1, 1, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="3-D"):
        tk.rotary(x[0], torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))


def test_overlap_and_span():
    def span(t):
        return _step._span(t.data_ptr(), t.shape, t.stride(), t.element_size())

    x = torch.zeros(64)
    assert span(x[8:16]) == (x.data_ptr() + 32, x.data_ptr() + 64)
    assert span(x.view(8, 8)[2:4, 1:3]) == (x.data_ptr() + 4 * 17, x.data_ptr() + 4 * 27)
    assert _step._overlap(span(x[:10]), span(x[9:])) and not _step._overlap(span(x[:9]), span(x[9:]))
    assert not _step._overlap(span(x[:0]), span(x))
    wide = torch.zeros((1, 4)).expand(3, 4)
    with pytest.raises(ValueError, match="broadcast"):
        _step._no_broadcast(wide.shape, wide.stride(), "out")
    _step._no_broadcast((1, 4), (0, 1), "out")


def test_packed_arguments_are_the_struct():
    """The bytes that a call packs are those of its ctypes Structure."""
    for kind, call in ((_step._RotaryArgs, _step._rotary), (_step._ScoresArgs, _step._scores),
                       (_step._AttentionArgs, _step._attention)):
        values = []
        for i, (_, t) in enumerate(kind._fields_):
            values.append(i + 0.5 if t is ctypes.c_float else 1000003 * (i + 1))
        packed = call.pack(*values)
        assert bytes(kind(*values)) == packed


def test_rotary_frequencies():
    plain = tk.rotary_frequencies(64, 10000.0, device="cpu")
    assert plain.dtype == torch.float64 and plain.shape == (32,)
    for i in (0, 1, 17, 31):
        assert plain[i].item() == pytest.approx(10000.0 ** (-2 * i / 64), rel=1e-14)
    linear = tk.rotary_frequencies(64, 10000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(linear * 4.0, plain, rtol=1e-15)
    based = tk.rotary_frequencies(64, 10000.0, scaling="base", factor=4.0, device="cpu")
    assert based[0] == 1.0 and based[-1].item() == pytest.approx(plain[-1].item() / 4.0, rel=1e-12)
    ramp = tk.rotary_frequencies(64, 10000.0, scaling="ramp", factor=4.0, original_length=4096, device="cpu")
    turns = plain * 4096 / (2 * math.pi)
    assert torch.equal(ramp[turns > 34], plain[turns > 34])
    assert torch.allclose(ramp[turns < 0.8] * 4.0, plain[turns < 0.8], rtol=1e-15)
    ratio = ramp / plain
    assert (ratio[1:] <= ratio[:-1] + 1e-15).all() and ratio[0] == 1.0 and ratio[-1].item() == pytest.approx(0.25)
    for wrong in (dict(rotated=3), dict(rotated=0), dict(rotated=8, base=0.0), dict(rotated=8, factor=0.5),
                  dict(rotated=8, scaling="other"), dict(rotated=2, scaling="base", factor=2.0),
                  dict(rotated=8, scaling="ramp", original_length=0), dict(rotated=8, scaling="ramp", fast=1.0),
                  dict(rotated=8, scaling="ramp", base=1.0)):
        with pytest.raises(ValueError):
            tk.rotary_frequencies(device="cpu", **wrong)


def test_turns_in_fixed_point():
    """The kernel's angle, in Python's integers: the mantissa times round(2^66
    / 2 pi), shifted, is the rate in turns to 2^-64 turns and the rounding of
    the constant (2^-64 relative)."""
    c = 0xa2f9836e4e44152a
    two_pi = 6.283185307179586476925286766559005768394
    for f in (1.0, 0.25, 1e-4, 3.7e-9, 2.5, 1000.0, 0.9999999):
        m, e = math.frexp(f)
        mantissa, biased = int(m * 2 ** 53), e + 1022
        turns = ((mantissa * c) >> (1077 - biased)) % 2 ** 64
        from fractions import Fraction

        want = Fraction(f) / Fraction(two_pi) % 1
        got = Fraction(turns, 2 ** 64)
        gap = abs(got - want)
        assert min(gap, 1 - gap) < Fraction(1, 2 ** 63) + Fraction(f) * Fraction(1, 2 ** 52)  # two_pi itself is a double
