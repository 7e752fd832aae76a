"""The operators of a paged cache in 8 bits on the host: refusals of the C entry points and of the binding, and the
formulas' own arithmetic."""

import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import cache_reference as C  # noqa: E402
import sparse_attention_indexer_fp32_gb300 as tk  # noqa: E402
from sparse_attention_indexer_fp32_gb300 import _cache  # noqa: E402
from test_step_host import SOME, _status, lib  # noqa: E402, F401

APPEND = dict(k=SOME, k_token_stride=128, k_head_stride=64, v=SOME, v_token_stride=128, v_head_stride=64, k_cache=SOME,
              k_cache_page_stride=2048, k_cache_token_stride=128, k_cache_head_stride=64, v_cache=SOME,
              v_cache_page_stride=2048, v_cache_token_stride=128, v_cache_head_stride=64, k_scales=SOME, v_scales=SOME,
              positions=SOME, frequencies=SOME, slots=SOME, num_pages=4, page_size=16, blocks=2, T=2, H=2, D=64, Dv=64,
              rotated=64, offset=0, layout=0, type=0, cache_type=3, scale=1.0)


def test_append_refusals(lib):  # noqa: F811
    bad = [dict(type=3), dict(type=-1), dict(cache_type=1), dict(cache_type=4), dict(T=-1), dict(H=-1), dict(H=65536),
           dict(D=0), dict(D=1025), dict(Dv=0), dict(Dv=1025), dict(rotated=-2), dict(rotated=33), dict(rotated=66),
           dict(offset=2), dict(offset=-2, rotated=32), dict(layout=2), dict(scale=math.inf), dict(scale=math.nan),
           dict(num_pages=-1), dict(page_size=-1), dict(blocks=0), dict(blocks=3), dict(blocks=-2), dict(blocks=32),
           dict(num_pages=2 ** 60), dict(k=None), dict(k_cache=None), dict(v_cache=None), dict(slots=None),
           dict(positions=None), dict(frequencies=None), dict(k_scales=None), dict(v_scales=None), dict(k=SOME + 1),
           dict(v=SOME + 1), dict(slots=SOME + 2), dict(positions=SOME + 2), dict(positions=SOME + 4, positions_64=1),
           dict(frequencies=SOME + 4), dict(k_scales=SOME + 2), dict(v_scales=SOME + 2),
           dict(cache_type=0, k_cache=SOME + 1), dict(cache_type=0, v_cache=SOME + 1), dict(type=2, k=SOME + 2)]
    for change in bad:
        assert _status(lib, "sparse_append", _cache._AppendArgs, APPEND, **change) == tk.Status.EINVAL, change
    for change in (dict(T=0), dict(H=0), dict(num_pages=0), dict(page_size=0), dict(T=0, k=None)):
        assert _status(lib, "sparse_append", _cache._AppendArgs, APPEND, **change) == tk.Status.OK, change
    assert lib.sparse_append(None, None) == tk.Status.EINVAL


def test_packed_arguments_are_the_struct():
    for kind, call in ((_cache._AppendArgs, _cache._append),):
        values = [i + 0.5 if t is ctypes.c_float else 1000003 * (i + 1) for i, (_, t) in enumerate(kind._fields_)]
        assert bytes(kind(*values)) == call.pack(*values)


def test_binding_refuses_tensors_off_the_gpu():
    k = torch.zeros((2, 2, 8), dtype=torch.bfloat16)
    n, cache = torch.zeros(2, dtype=torch.int32), torch.zeros((1, 4, 2, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        tk.cache_append(k, k, n, torch.zeros(4, dtype=torch.float64), cache, cache.clone(), n)
    with pytest.raises(ValueError, match="k requires a gradient"):
        tk.cache_append(k.requires_grad_(), None, None, None, cache, None, n)


def test_caches_side_by_side():
    """Parts of one tensor share no element; caches that share one, or whose addresses mix otherwise, are refused."""

    def meet(a, b):
        return _cache._meet(a.shape, a.stride(), b.stride(), b.shape[3], b.data_ptr() - a.data_ptr(), a.element_size())

    t = torch.zeros((5, 2, 4, 3, 8))
    assert not meet(t[:, 0], t[:, 1]) and not meet(t[:, 1], t[:, 0])
    assert meet(t[:, 0], t[:, 0])
    t = torch.zeros((5, 4, 3, 20))
    assert not meet(t[..., :8], t[..., 8:]) and not meet(t[..., 8:], t[..., :8]) and not meet(t[..., :8], t[..., 12:])
    assert meet(t[..., :8], t[..., 7:]) and meet(t[..., 7:], t[..., :8])
    t = torch.zeros((5, 3, 4, 20)).transpose(1, 2)
    assert not meet(t[..., :8], t[..., 8:]) and meet(t[..., :9], t[..., 8:])
    t = torch.zeros((6, 4, 3, 8))
    assert not meet(t[:3], t[3:]) and meet(t[:4], t[2:]) and not meet(t[0::2], t[1::2])
    assert meet(t[:3], t.view(6, 3, 4, 8).transpose(1, 2)[:3])


def test_rounding_of_the_reference():
    """The reference's rounding is torch's, for every code, every border between two and what lies past the ends."""
    codes = np.sort(C.VALUES[np.isfinite(C.VALUES)])
    mids = (codes[1:] + codes[:-1]) / 2
    x = np.concatenate([codes, mids, np.nextafter(mids, 1e9), np.nextafter(mids, -1e9), [463.0, 500.0, 1e30, -1e30]])
    with_torch = torch.from_numpy(x).clamp(-448.0, 448.0).float()
    exact = with_torch.double().numpy() == np.clip(x, -448.0, 448.0)  # a border's neighbours are no float32
    assert np.array_equal(C.round_e4m3(x)[exact], with_torch.to(C.E4M3).double().numpy()[exact])
    assert np.isnan(C.round_e4m3([np.nan, np.inf, -np.inf])).all()
    for most, want in ((0.0, 2.0 ** -126), (448.0, 1.0), (448.1, 2.0), (3.5, 2.0 ** -7), (3.6, 2.0 ** -6), (1e38, 2.0 ** 118)):
        assert C.power_for(most) == want


ATTENTION = dict(q=SOME, q_seq_stride=256, q_token_stride=256, q_head_stride=64, k=SOME, k_page_stride=2048,
                 k_token_stride=128, k_head_stride=64, v=SOME, v_page_stride=2048, v_token_stride=128,
                 v_head_stride=64, indices=SOME, page_table=SOME, table_stride=4, table_width=4, out=SOME,
                 num_pages=8, page_size=16, B=2, T=1, Hq=4, Hkv=2, D=64, Dv=64, K=8, type=0, scale=0.125,
                 k_scales=SOME, v_scales=SOME, blocks=4)


def test_attention_refusals(lib):  # noqa: F811
    from sparse_attention_indexer_fp32_gb300 import _step

    most = 2 ** 31 - 1
    bad = [dict(type=2), dict(type=3), dict(B=-1), dict(T=-1), dict(Hkv=0), dict(Hq=3), dict(Hq=-2), dict(K=-1),
           dict(D=0), dict(D=72), dict(D=8), dict(D=272), dict(Dv=0), dict(Dv=8), dict(Dv=24), dict(Dv=272),
           dict(scale=math.nan), dict(scale=math.inf), dict(softcap=-1.0), dict(softcap=math.nan), dict(softcap=math.inf),
           dict(num_pages=-1), dict(page_size=-1), dict(table_width=-1), dict(table_stride=-1), dict(slopes=SOME),
           dict(page_table=None, first=SOME), dict(page_table=None, query_positions=SOME), dict(q=None), dict(k=None),
           dict(v=None), dict(indices=None), dict(out=None), dict(k=SOME + 8), dict(v=SOME + 8), dict(out=SOME + 8),
           dict(q=SOME + 1), dict(k_page_stride=2056), dict(k_token_stride=136), dict(k_head_stride=72),
           dict(v_page_stride=2056), dict(v_token_stride=136), dict(v_head_stride=72), dict(indices=SOME + 2),
           dict(page_table=SOME + 2), dict(query_positions=SOME + 2), dict(first=SOME + 2), dict(lse=SOME + 2),
           dict(slopes=SOME + 2, query_positions=SOME), dict(num_pages=2 ** 60), dict(k_scales=None),
           dict(v_scales=None), dict(k_scales=SOME + 2), dict(v_scales=SOME + 2), dict(blocks=0), dict(blocks=3),
           dict(blocks=-4), dict(blocks=32), dict(B=most, T=most), dict(B=2 ** 30, T=1, Hkv=4),
           dict(B=2 ** 12, T=1, Hkv=1, Hq=most)]
    for change in bad:
        assert _status(lib, "sparse_attention_e4m3", _step._AttentionE4m3Args, ATTENTION, **change) == tk.Status.EINVAL, change
    for change in (dict(B=0), dict(T=0), dict(Hq=0)):
        assert _status(lib, "sparse_attention_e4m3", _step._AttentionE4m3Args, ATTENTION, **change) == tk.Status.OK, change
    assert lib.sparse_attention_e4m3(None, None) == tk.Status.EINVAL
    kind, call = _step._AttentionE4m3Args, _step._attention_e4m3
    values = [i + 0.5 if t is ctypes.c_float else 1000003 * (i + 1) for i, (_, t) in enumerate(kind._fields_)]
    packed = call.pack(*values)
    assert bytes(kind(*values))[:len(packed)] == packed or bytes(kind(*values)) == packed


def test_scales_are_checked():
    """Scales of another shape, or blocks that do not divide the page, are refused by name before anything else of them."""
    from sparse_attention_indexer_fp32_gb300 import _step

    for scales in (None, torch.zeros((2, 3)), torch.zeros((2, 0, 4)), torch.zeros((2, 3, 4))):
        with pytest.raises(ValueError, match="k_scales must be"):
            _step._scales_of(scales, "k_scales", 2, 16, 4, 0)
    with pytest.raises(ValueError, match="contiguous"):
        _step._scales_of(torch.zeros((2, 4, 4)), "k_scales", 2, 16, 4, 0)  # not on the GPU


def test_addresses_behind_the_last_element():
    for t in (torch.zeros((3, 4, 8)), torch.zeros((3, 4, 8, 2)), torch.zeros((5, 6, 7))[1:4, ::2, 2:5], torch.zeros((3, 0, 8)),
              torch.zeros((4, 1, 2, 9)).transpose(0, 2)):
        want = t.data_ptr() + 4 * (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) if t.numel() else t.data_ptr()
        assert _cache._end(t.data_ptr(), t.shape, t.stride(), 4) == want
