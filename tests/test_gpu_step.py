"""The operators around the selection on the GPU against their formulas in 64
bits (``step_reference``): types, layouts, odd sizes, strides, lengths from
nothing to past the width, masks that leave a row empty, NaN where nothing may
be read, pages outside the cache, other streams and captured graphs."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_attention_indexer_fp32_gb300 as tk  # noqa: E402

DEV = torch.device("cuda:0")
BF16, FP16, FP32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, seed, dtype=FP32, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * scale).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# ---- rotary ------------------------------------------------------------------------------------------

ROTARY = [
    # T, H, D, rotated, offset, layout, dtype
    (1, 1, 2, 2, 0, "half", BF16),
    (1, 64, 128, 64, 0, "half", BF16),
    (4, 64, 128, 64, 64, "interleaved", BF16),
    (5, 3, 80, 80, 0, "interleaved", FP32),
    (3, 7, 96, 32, 8, "half", FP16),
    (3, 2, 20, 6, 5, "half", BF16),  # nothing aligned: a pair at a time
    (3, 2, 20, 6, 5, "interleaved", FP32),
    (2, 3, 33, 32, 1, "interleaved", FP16),
    (700, 1, 128, 128, 0, "half", BF16),  # one head: the table bounds the tokens of a CTA
    (301, 33, 64, 64, 0, "half", FP32),
    (2500, 16, 128, 64, 0, "interleaved", BF16),  # several items a thread
    (2, 2, 1024, 1024, 0, "half", FP32),
    (1, 2, 1022, 1022, 0, "half", BF16),
]


@pytest.mark.parametrize("T,H,D,rotated,offset,layout,dtype", ROTARY)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(T, H, D, rotated, offset, layout, dtype, inverse):
    x = _randn((T, H, D), T * H + D, dtype)
    pos = torch.randint(-5, 1 << 20, (T,), generator=_gen(1), device=DEV).to(torch.int32)
    f = tk.rotary_frequencies(rotated, 10000.0, device=DEV)
    kw = dict(layout=layout, offset=offset, scale=1.25, inverse=inverse)
    want, bound = R.rotary(x, pos, f, layout, offset, 1.25, inverse)
    R.assert_near(tk.rotary(x, pos, f, **kw), want, bound, "out of place")
    R.assert_near(tk.rotary(x, pos.long(), f, **kw), want, bound, "64-bit positions")
    # in place, in a slice of a joint tensor: the neighbours stay
    joint = torch.full((T, H + 2, D), 7.0, dtype=dtype, device=DEV)
    joint[:, 1:-1] = x
    view = joint[:, 1:-1]
    assert tk.rotary(view, pos, f, out=view, **kw) is view
    R.assert_near(view, want, bound, "in place")
    assert (joint[:, 0] == 7.0).all() and (joint[:, -1] == 7.0).all()


def test_rotary_far_positions_and_rates():
    """Positions to both ends of 32 bits, and past them in 64; rates under and
    over a turn a position, zero and negative."""
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int64, device=DEV)
    f = torch.tensor([1.0, 0.0, -0.5, 7.75, 1e-9, 1e-300, 3.0e5, 0.1], dtype=torch.float64, device=DEV)
    x = _randn((6, 2, 16), 3)
    got = tk.rotary(x, pos.to(torch.int32), f)
    # the rate's rounding to 2^-64 turns and the double's own to 2^-53, times the position
    want, bound = R.rotary(x, pos, f, "half", 0, 1.0, False)
    drift = pos.abs().double() * 2.0 ** -62 * 7
    more = np.abs(R.np64(x)).sum(-1, keepdims=True) * R.np64(drift)[:, None, None]
    R.assert_near(got, want, bound + more)
    assert torch.equal(tk.rotary(x, pos, f), got)


def test_rotary_backward_is_the_inverse():
    """The gradient against differences: <dy, J dx> = <J' dy, dx> for random
    directions, and the round trip."""
    T, H, D = 9, 4, 64
    f = tk.rotary_frequencies(48, device=DEV)
    pos = _ints(list(range(100, 100 + T)))
    x, dx, dy = (_randn((T, H, D), s) for s in (1, 2, 3))
    kw = dict(offset=8, scale=0.75, layout="interleaved")
    moved = tk.rotary(x + dx, pos, f, **kw).double() - tk.rotary(x, pos, f, **kw).double()
    grad = tk.rotary(dy, pos, f, inverse=True, **kw).double()
    # three results rounded to FP32 and the trigonometric bound, over T H D terms
    scale = (moved.abs() * dy.abs()).sum() + (grad.abs() * dx.abs()).sum() + (x.abs() * dy.abs()).sum().double()
    assert abs((moved * dy).sum() - (grad * dx).sum()) <= 64 * R.U * scale
    kw["scale"] = 1.0
    back = tk.rotary(tk.rotary(x, pos, f, **kw), pos, f, inverse=True, **kw)
    assert (back - x).abs().max() <= 64 * R.U * x.abs().max()


@pytest.mark.parametrize("dtype,D,pad", [(BF16, 128, 0), (FP32, 24, 4), (FP16, 18, 0)])
def test_rotary_into_a_paged_cache(dtype, D, pad):
    """Tokens without a slot, or with one past the cache, are not written, and
    nothing else of the cache changes."""
    T, H, pages, ps = 21, 3, 5, 7
    x = _randn((T, H, D), 5, dtype)
    f = tk.rotary_frequencies(D - D % 4, device=DEV)
    pos = _ints(list(range(T)))
    slots = torch.randperm(pages * ps, generator=_gen(2), device=DEV)[:T].to(torch.int32)
    slots[3], slots[8], slots[9], slots[20] = -1, pages * ps, 2 ** 31 - 1, -2 ** 31
    cache = torch.full((pages, ps, H, D + pad), -3.0, dtype=dtype, device=DEV)
    view = cache[..., :D]
    tk.rotary(x, pos, f, out=view, slots=slots)
    want, bound = R.rotary(x, pos, f, "half", 0, 1.0, False)
    full, fb = np.full((pages * ps, H, D), -3.0), np.zeros((pages * ps, H, D))
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * ps:
            full[s], fb[s] = want[t], bound[t]
    R.assert_near(view, full.reshape(view.shape), fb.reshape(view.shape))
    assert (cache[..., D:] == -3.0).all()


def test_rotary_nothing_to_do():
    f = tk.rotary_frequencies(8, device=DEV)
    assert tk.rotary(torch.empty((0, 2, 8), device=DEV), _ints([]), f).shape == (0, 2, 8)
    assert tk.rotary(torch.empty((2, 0, 8), device=DEV), _ints([1, 2]), f).shape == (2, 0, 8)
    cache = torch.empty((0, 4, 2, 8), device=DEV)
    tk.rotary(torch.zeros((2, 2, 8), device=DEV), _ints([1, 2]), f, out=cache, slots=_ints([0, 1]))


# ---- indexer scores ----------------------------------------------------------------------------------


def _scores_case(B, T, H, D, width, ps, dtype, lengths, seed=0, pad=0, extra=2):
    pages = -(-width // ps)
    total = B * pages + extra
    table = torch.randperm(total, generator=_gen(seed), device=DEV)[:B * pages].to(torch.int32).view(B, pages)
    e4m3 = dtype == E4M3
    pool = _randn((total, ps, D + pad), seed + 1, FP32, 3.0 if e4m3 else 1.0).to(dtype)
    scales = torch.rand((total, ps), generator=_gen(seed + 2), device=DEV) + 0.5 if e4m3 else None
    q = _randn((B, T, H, D), seed + 3).to(dtype)
    w = _randn((B, T, H), seed + 4)
    n = _ints(lengths).view(B, T)
    return q, w, pool[..., :D], n, table, scales


def _check_scores(args, width, **kw):
    q, w, keys, n, table, scales = args
    out = torch.full((q.shape[0], q.shape[1], width), 12345.0, device=DEV)
    tk.indexer_scores(q, w, keys, n, table, key_scales=scales, out=out, **kw)
    want, bound = R.scores(q, w, keys, n, table, scales, width)
    unwritten = np.isnan(want) & (R.np64(out) == 12345.0)
    want[unwritten] = 12345.0
    R.assert_near(out, want, bound)
    return out


SCORES = [
    # B, T, H, D, width, page_size, dtype, lengths
    (1, 1, 1, 8, 1, 1, BF16, [1]),
    (4, 1, 64, 128, 1000, 64, BF16, [0, 300, 1000, 64]),
    (2, 3, 32, 128, 517, 16, E4M3, [517, 516, 515, 1, 0, -7]),
    (3, 1, 7, 64, 129, 5, FP16, [128, 129, 2000]),
    (2, 1, 128, 128, 700, 64, BF16, [700, 333]),
    (1, 1, 24, 40, 300, 48, BF16, [257]),
    (1, 1, 5, 48, 300, 300, E4M3, [299]),
    (1, 37, 64, 128, 400, 64, BF16, list(range(364, 401))),
    (2, 9, 33, 96, 260, 64, FP16, [260] * 9 + list(range(120, 129))),
    (1, 130, 8, 64, 300, 32, E4M3, [(7 * i) % 301 for i in range(130)]),
    (1, 3, 96, 128, 2500, 64, BF16, [2500, 1300, 900]),
    (1, 100, 1, 128, 200, 64, BF16, [(3 * i) % 201 for i in range(100)]),
    (2, 45, 8, 64, 300, 64, FP16, [300 - i for i in range(90)]),
    (1, 33, 3, 32, 140, 16, E4M3, [140 - i for i in range(33)]),
    (2, 17, 16, 128, 260, 64, BF16, [260 - 2 * i for i in range(34)]),
    (3, 2, 10, 64, 1300, 7, BF16, [1300, 1299, 5, 4, 700, 0]),
    (1, 2, 64, 128, 128 * 40 + 1, 128, FP16, [128 * 40 + 1, 128 * 40]),
]


@pytest.mark.parametrize("B,T,H,D,width,ps,dtype,lengths", SCORES)
def test_scores(B, T, H, D, width, ps, dtype, lengths):
    _check_scores(_scores_case(B, T, H, D, width, ps, dtype, lengths), width)


@pytest.mark.parametrize("B,T,H,D,ps,dtype", [(330, 1, 32, 64, 64, BF16), (120, 3, 64, 64, 16, FP16),
                                              (330, 1, 16, 64, 7, BF16), (40, 70, 2, 64, 64, BF16), (150, 2, 70, 128, 128, E4M3)])
def test_scores_many_units_per_cta(B, T, H, D, ps, dtype):
    """Several work units of many tiles on every CTA, ragged, some empty."""
    width = 2300
    lengths = torch.randint(-100, width + 50, (B, T), generator=_gen(B), device=DEV).flatten().tolist()
    args = _scores_case(B, T, H, D, width, ps, dtype, lengths)
    first = _check_scores(args, width)
    for _ in range(3):
        assert torch.equal(_check_scores(args, width) if _ == 0 else tk.indexer_scores(
            *args[:5], key_scales=args[5], out=torch.full_like(first, 12345.0)), first)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_scores_strides(dtype):
    """Padded keys, queries that are a slice (at an odd element), broadcast
    page tables, an output with longer rows."""
    B, T, H, D, width, ps = 3, 2, 12, 64, 333, 16
    q, w, keys, n, table, scales = _scores_case(B, T, H, D, width, ps, dtype, [333, 332, 17, 16, 200, 199], pad=32)
    joint = torch.zeros((B, T, H, D + 5), dtype=FP32, device=DEV).to(dtype)
    joint[..., 1:D + 1] = q
    table = table[:1].expand(B, -1)
    long = torch.full((B, T, width + 9), 5.0, device=DEV)
    got = tk.indexer_scores(joint[..., 1:D + 1], w, keys, n, table, key_scales=scales, out=long[..., :width])
    assert (long[..., width:] == 5.0).all()
    want, bound = R.scores(q, w, keys, n, table, scales, width)
    keep = ~np.isnan(want)
    R.assert_near(R.np64(got)[keep], want[keep], bound[keep])


def test_scores_values_that_are_not_read():
    """Pages outside the cache give -inf; what lies past a length, and the
    cache's other entries, may hold NaN."""
    q, w, keys, n, table, _ = _scores_case(2, 1, 16, 64, 260, 16, BF16, [250, 100])
    keys = keys.contiguous()
    used = torch.zeros(keys.shape[0] * 16, dtype=torch.bool, device=DEV)
    for b, m in enumerate((250, 100)):
        s = torch.arange(m, device=DEV)
        used[(table[b].long()[s // 16] * 16 + s % 16)] = True
    keys.view(-1, 64)[~used] = math.nan
    table[0, 3], table[0, 5], table[1, 0] = -1, keys.shape[0], 2 ** 31 - 1
    out = _check_scores((q, w, keys, n, table, None), 260)
    assert torch.isneginf(out[0, 0, 48:64]).all() and torch.isneginf(out[1, 0, :16]).all()
    assert torch.isfinite(out[0, 0, :48]).all()


def test_scores_keep_nan_and_infinities():
    q, w, keys, n, table, _ = _scores_case(1, 1, 8, 64, 64, 64, BF16, [64])
    keys = keys.contiguous()
    w = w.abs() + 0.1
    keys[table[0, 0].long(), 5] = math.nan
    got = tk.indexer_scores(q, w, keys, n, table)
    assert torch.isnan(got[0, 0, 5]) and torch.isfinite(got[0, 0, :5]).all() and torch.isfinite(got[0, 0, 6:]).all()


def test_scores_feed_the_selection():
    """The indices that the scores select are those of the formula wherever
    its values are further apart than the bound."""
    B, width, k = 6, 5000, 512
    args = _scores_case(B, 1, 64, 128, width, 64, BF16, [5000, 4000, 511, 0, 513, 4999])
    out = tk.indexer_scores(*args[:5])
    idx = tk.topk_ragged(out.view(B, -1), args[3].view(-1), k).cpu().numpy()
    want, bound = R.scores(*args, out.shape[2])
    for b in range(B):
        m = int(args[3][b, 0])
        got = idx[b][idx[b] >= 0]
        assert len(got) == min(m, k)
        left = np.setdiff1d(np.arange(m), got)
        if len(left) and len(got):
            assert (want[b, 0, got] + bound[b, 0, got]).min() >= (want[b, 0, left] - bound[b, 0, left]).max()


def test_scores_nothing_to_do():
    q, w, keys, n, table, _ = _scores_case(1, 1, 8, 64, 64, 64, BF16, [64])
    assert tk.indexer_scores(q[:0], w[:0], keys, n[:0], table[:0]).shape == (0, 1, 64)
    assert tk.indexer_scores(q, w, keys, n, table, width=0).shape == (1, 1, 0)
    empty = tk.indexer_scores(q, w, keys[:0], n, table)  # every page lies outside a cache of none
    assert torch.isneginf(empty).all()
    none = torch.empty((0, 64, 64), dtype=BF16, device=DEV)  # and without an address
    assert torch.isneginf(tk.indexer_scores(q, w, none, n, table)).all()


# ---- attention ---------------------------------------------------------------------------------------


def _attention_case(B, T, Hq, Hkv, D, Dv, K, S, ps, dtype, seed=0, shared=False, sel="random", pad=0):
    pages = -(-S // ps)
    total = B * pages + 2
    table = torch.randperm(total, generator=_gen(seed), device=DEV)[:B * pages].to(torch.int32).view(B, pages)
    kp = _randn((total, ps, Hkv, D + pad), seed + 1, dtype)
    k = kp[..., :D]
    v = k[..., :Dv] if shared else _randn((total, ps, Hkv, Dv), seed + 2, dtype)
    q = _randn((B, T, Hq, D), seed + 3, dtype, 1.5)
    r = torch.rand((B, T, S), generator=_gen(seed + 4), device=DEV)
    indices = r.topk(min(K, S), dim=-1).indices.sort(dim=-1).values.to(torch.int32)
    if K > S:
        indices = torch.cat([indices, torch.full((B, T, K - S), -1, dtype=torch.int32, device=DEV)], dim=-1)
    if sel == "holes":  # empty slots anywhere, a row of none, a row of one
        indices = torch.where(torch.rand((B, T, K), generator=_gen(seed + 5), device=DEV) < 0.4, -1, indices)
        indices[0, 0] = -1
        indices[-1, -1, 1:] = -1
        indices[-1, -1, 0] = S // 2
    return q, k, v, indices.contiguous(), table


def _check_attention(q, k, v, indices, table, query_positions=None, softcap=0.0, slopes=None, first=None, scale=None):
    got, lse = tk.sparse_attention(q, k, v, indices, table, query_positions=query_positions, softcap=softcap,
                                   slopes=slopes, first=first, scale=scale, return_lse=True)
    want = R.attention(q, k, v, indices, table, query_positions, q.shape[3] ** -0.5 if scale is None else scale,
                       softcap, slopes, first)
    R.assert_near(got, want[0], want[1], "out")
    R.assert_near(lse, want[2], want[3], "lse")
    return got, lse


ATTENTION = [
    # B, T, Hq, Hkv, D, Dv, K, S, page_size, dtype, shared, selection
    (1, 1, 1, 1, 8, 8, 1, 1, 1, BF16, False, "random"),
    (2, 1, 32, 4, 128, 128, 512, 900, 64, BF16, False, "random"),
    (2, 2, 16, 2, 64, 64, 77, 200, 16, FP16, False, "holes"),
    (1, 3, 10, 5, 96, 64, 130, 300, 17, FP16, False, "holes"),
    (1, 2, 64, 1, 256, 192, 200, 400, 64, BF16, True, "random"),
    (1, 1, 128, 1, 256, 256, 129, 300, 64, BF16, False, "holes"),
    (1, 1, 150, 1, 64, 128, 64, 128, 32, FP16, False, "random"),  # more heads than one tile of 128 rows
    (2, 1, 40, 1, 128, 64, 65, 100, 64, BF16, True, "holes"),
    (1, 1, 70, 1, 192, 192, 300, 400, 48, FP16, True, "holes"),
    (1, 1, 8, 8, 128, 128, 1, 50, 64, BF16, False, "random"),
    (3, 1, 4, 1, 40, 24, 63, 64, 3, BF16, False, "holes"),
    (1, 1, 8, 2, 128, 128, 2048, 3000, 64, BF16, False, "random"),
    (2, 1, 8, 1, 128, 128, 100, 60, 16, FP16, False, "random"),  # more slots than positions
    (1, 1, 6, 2, 256, 8, 40, 60, 16, BF16, False, "random"),
    (1, 1, 40, 1, 256, 256, 130, 300, 64, FP16, False, "holes"),  # two copies, two stages
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,Dv,K,S,ps,dtype,shared,sel", ATTENTION)
def test_attention(B, T, Hq, Hkv, D, Dv, K, S, ps, dtype, shared, sel):
    _check_attention(*_attention_case(B, T, Hq, Hkv, D, Dv, K, S, ps, dtype, shared=shared, sel=sel))


@pytest.mark.parametrize("rows,Hq,Hkv,D,Dv,K,shared", [(340, 40, 1, 64, 64, 130, False), (340, 70, 1, 64, 48, 64, True),
                                                       (170, 80, 2, 128, 64, 190, False), (500, 36, 1, 128, 128, 1, True),
                                                       (400, 8, 1, 64, 64, 70, False)])
def test_attention_many_rows_per_cta(rows, Hq, Hkv, D, Dv, K, shared):
    """More rows than places for CTAs, odd numbers of tiles, empty rows between
    full ones; cap, bias and masks change from row to row."""
    S = 300
    q, k, v, idx, table = _attention_case(1, rows, Hq, Hkv, D, Dv, K, S, 16, BF16, shared=shared, sel="holes")
    idx[0, ::7] = -1
    qpos = torch.randint(0, S, (1, rows), generator=_gen(9), device=DEV).to(torch.int32)
    first = torch.randint(-5, S // 2, (1, rows), generator=_gen(10), device=DEV).to(torch.int32)
    slopes = torch.rand(Hq, generator=_gen(11), device=DEV) * 0.05
    got = _check_attention(q, k, v, idx, table, query_positions=qpos, softcap=20.0, slopes=slopes, first=first)
    again = tk.sparse_attention(q, k, v, idx, table, query_positions=qpos, softcap=20.0, slopes=slopes, first=first,
                                return_lse=True)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    _check_attention(q, k, v, idx[:, :, :0].contiguous(), table)


@pytest.mark.parametrize("cap,biased,masked", [(30.0, False, False), (0.0, True, False), (5.0, True, True),
                                               (0.0, False, True)])
@pytest.mark.parametrize("Hq,Hkv", [(12, 3), (96, 1)])
def test_attention_cap_bias_and_masks(cap, biased, masked, Hq, Hkv):
    B, T, S, K = 3, 2, 500, 150
    q, k, v, idx, table = _attention_case(B, T, Hq, Hkv, 64, 64, K, S, 16, BF16, sel="holes")
    qpos = _ints([[499, 498], [250, 249], [0, 499]])
    slopes = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=FP32) / Hq) if biased else None
    first = _ints([[0, 498], [100, 251], [0, -3]]) if masked else None  # [1, 1]: starts past the query, sees nothing
    got, lse = _check_attention(q, k, v, idx, table, query_positions=qpos, softcap=cap, slopes=slopes, first=first)
    if masked:
        assert (got[1, 1] == 0).all() and torch.isneginf(lse[1, 1]).all()


def test_attention_takes_slots_and_strides():
    """Without a page table the indices are slots (topk_paged); queries that
    are a slice at an odd element, padded entries, broadcast page tables."""
    q, k, v, idx, table = _attention_case(2, 2, 16, 4, 64, 64, 90, 300, 16, BF16, sel="holes", pad=8)
    table = table[:1].expand(2, -1)
    want = tk.sparse_attention(q, k, v, idx, table)
    joint = torch.zeros((2, 2, 16, 64 + 3), dtype=BF16, device=DEV)
    joint[..., 1:65] = q
    assert torch.equal(tk.sparse_attention(joint[..., 1:65], k, v, idx, table), want)
    pages = torch.gather(table.long(), 1, idx.clamp(min=0).flatten(1).long() // 16).view(idx.shape)
    slots = torch.where(idx < 0, -1, pages.int() * 16 + idx % 16).int().contiguous()
    assert torch.equal(tk.sparse_attention(q, k, v, slots, None), want)
    _check_attention(q, k, v, slots, None)
    by_head = k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)  # heads before tokens in a page
    assert torch.equal(tk.sparse_attention(q, by_head, v, idx, table), want)


@pytest.mark.parametrize("shared", [False, True])
def test_attention_values_that_are_not_read(shared):
    """Everything that no row sees holds NaN or infinities; pages and
    positions outside the table or the cache count as absent."""
    B, S, K, ps = 2, 256, 100, 16
    q, k, v, idx, table = _attention_case(B, 1, 8, 2, 64, 64, K, S, ps, BF16, sel="holes", shared=shared)
    idx[1, 0, 0], idx[1, 0, 1], idx[1, 0, 2] = 2 ** 31 - 1, S, -2 ** 31
    k = k.contiguous()
    v = k[..., :64] if shared else v.contiguous()
    qpos, first = _ints([[S], [200]]), _ints([[0], [50]])
    seen = torch.zeros(k.shape[0] * ps, dtype=torch.bool, device=DEV)
    for b in range(B):
        p = idx[b, 0].long()
        p = p[(p >= 0) & (p < S)]
        p = p[(p <= int(qpos[b])) & (p >= int(first[b]))]
        seen[table[b].long()[p // ps] * ps + p % ps] = True
    k.view(-1, 2, k.shape[3])[~seen] = math.nan
    if not shared:
        v.view(-1, 2, 64)[~seen] = math.inf
    table[1, 7], table[1, 8] = -1, k.shape[0]
    got, _ = _check_attention(q, k, v, idx, table, query_positions=qpos, first=first)
    assert torch.isfinite(got).all()


def test_attention_large_logits():
    """Logits of thousands, of either sign, growing along the list: the
    running maximum moves by more than an exponent's range."""
    q, k, v, idx, table = _attention_case(1, 1, 4, 1, 64, 64, 700, 800, 16, BF16)
    k = (k * torch.linspace(0, 60, k.shape[0], device=DEV)[:, None, None, None]).to(BF16)
    _check_attention(q, k, v, idx, table, scale=1.0)
    _check_attention(q, k, v, idx, table, scale=-1.0)
    _check_attention(q, k, v, idx, table, scale=0.0)


def test_attention_nothing_to_do():
    q, k, v, idx, table = _attention_case(2, 1, 4, 2, 64, 64, 10, 50, 16, BF16)
    out, lse = tk.sparse_attention(q, k, v, idx[..., :0].contiguous(), table, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = tk.sparse_attention(q, k[:0], v[:0], idx, table, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    none = torch.empty((0, 16, 2, 64), dtype=BF16, device=DEV)
    assert (tk.sparse_attention(q, none, none, idx, table) == 0).all()
    assert tk.sparse_attention(q[:0], k, v, idx[:0], table[:0]).shape == (0, 1, 4, 64)


# ---- streams, graphs, repeatability ------------------------------------------------------------------


def _step(q_in, pos, f, idx_q, w, ikeys, kcache, vcache, n, table, k_sel, bufs):
    """A step as a program runs it: rotate, score, select, attend."""
    q = tk.rotary(q_in, pos, f, out=bufs["q"])
    B = n.shape[0]
    scores = tk.indexer_scores(idx_q, w, ikeys, n, table, out=bufs["scores"])
    idx = tk.topk_ragged(scores.view(B, -1), n.view(-1), k_sel, out=bufs["idx"])
    return tk.sparse_attention(q.view(B, 1, *q.shape[1:]), kcache, vcache, idx.view(B, 1, -1), table,
                               query_positions=n - 1, out=bufs["out"])


def _step_inputs(B=3, S=1500, k_sel=256, seed=0):
    iq, w, ikeys, n, table, _ = _scores_case(B, 1, 32, 64, S, 16, BF16, [1500, 700, 100][:B], seed=seed)
    _, k, v, _, _ = _attention_case(B, 1, 16, 2, 64, 64, 8, S, 16, BF16, seed=seed + 10)
    q_in = _randn((B, 16, 64), seed + 20, BF16)
    pos = (n.view(-1) - 1).contiguous()
    bufs = dict(q=torch.empty_like(q_in), scores=torch.full((B, 1, S), -1.0, device=DEV),
                idx=torch.empty((B, k_sel), dtype=torch.int32, device=DEV),
                out=torch.empty((B, 1, 16, 64), dtype=BF16, device=DEV))
    return [q_in, pos, tk.rotary_frequencies(64, device=DEV), iq, w, ikeys, k, v, n, table, k_sel, bufs]


def test_step_on_another_stream_and_in_a_graph():
    args = _step_inputs()
    want = _step(*args).clone()
    side = torch.cuda.Stream()
    args[-1]["out"].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _step(*args)
    side.synchronize()
    assert torch.equal(args[-1]["out"], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(*args)
    other = _step_inputs(seed=77)
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 9):  # new inputs in the captured buffers
        args[i].copy_(other[i])
    args[8][0, 0], args[1][0] = 37, 36
    graph.replay()
    torch.cuda.synchronize()
    got = args[-1]["out"].clone()
    for b in args[-1].values():
        b.zero_()
    assert torch.equal(_step(*args), got)


def test_calls_take_their_stream_argument():
    args = _step_inputs()
    side = torch.cuda.Stream()
    x, pos, f = args[:3]
    want = tk.rotary(x, pos, f)
    out = torch.zeros_like(x)
    torch.cuda.synchronize()
    tk.rotary(x, pos, f, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_results_belong_to_the_calls_stream():
    """A result allocated by a call on another stream is that stream's memory:
    freed there, it is not handed to the current stream while in use."""
    x, f, pos = _randn((64, 8, 64), 1, BF16), tk.rotary_frequencies(64, device=DEV), _ints(list(range(64)))
    side = torch.cuda.Stream()
    want = tk.rotary(x, pos, f)
    torch.cuda.synchronize()
    got = tk.rotary(x, pos, f, stream=side)
    at = got.data_ptr()
    side.synchronize()
    assert torch.equal(got, want)
    del got
    assert torch.empty_like(x).data_ptr() != at  # the current stream's pool has other blocks


@pytest.mark.parametrize("ps", [64, 48])
def test_offsets_past_32_bits(ps):
    """Entries behind 2^32 elements of a cache (10 GB), by boxes and by copies."""
    pages = (1 << 32) // (ps * 128) + 64
    keys = torch.empty((pages, ps, 128), dtype=BF16, device=DEV)
    last = list(range(pages - 9, pages))
    table = _ints([last])
    keys[last[0]:] = _randn((9, ps, 128), 5, BF16)
    width = 8 * ps + 3
    q, w = _randn((1, 1, 8, 128), 6, BF16), _randn((1, 1, 8), 7)
    few = keys[last[0]:].contiguous()
    local = _ints([list(range(9))])
    n = _ints([[width]])
    assert torch.equal(tk.indexer_scores(q, w, keys, n, table, width=width), tk.indexer_scores(q, w, few, n, local, width=width))
    idx = torch.arange(width, dtype=torch.int32, device=DEV).view(1, 1, -1)
    cache, small = keys[:, :, None], few[:, :, None]
    assert torch.equal(tk.sparse_attention(q, cache, cache, idx, table), tk.sparse_attention(q, small, small, idx, local))
    if pages * ps < 2 ** 31:
        f, pos = tk.rotary_frequencies(128, device=DEV), _ints([5, 6])
        slots = _ints([pages * ps - 1, pages * ps - ps])
        tk.rotary(q[0, 0, :2, None], pos, f, out=cache, slots=slots)
        assert torch.equal(cache.view(-1, 1, 128)[slots.long()], tk.rotary(q[0, 0, :2, None], pos, f))


def test_attention_keeps_nan_that_is_seen():
    q, k, v, idx, table = _attention_case(1, 1, 8, 2, 64, 64, 100, 200, 16, BF16)
    p = int(idx[0, 0, 40])
    k[table[0, p // 16].long(), p % 16, 0] = math.nan
    out, lse = tk.sparse_attention(q, k, v, idx, table, return_lse=True)
    assert torch.isnan(out[0, 0, :4]).all() and torch.isnan(lse[0, 0, :4]).all()
    assert torch.isfinite(out[0, 0, 4:]).all() and torch.isfinite(lse[0, 0, 4:]).all()


def test_repeated_calls_agree():
    """Byte for byte, on a batch whose rows are split over several CTAs and on
    one that is not."""
    for B, K in ((1, 2048), (40, 300)):
        q, k, v, idx, table = _attention_case(B, 1, 32, 4, 128, 128, K, 2100, 64, BF16, sel="holes")
        first = tk.sparse_attention(q, k, v, idx, table, return_lse=True)
        for _ in range(20):
            again = tk.sparse_attention(q, k, v, idx, table, return_lse=True)
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    args = _scores_case(3, 1, 64, 128, 3000, 64, BF16, [3000, 100, 2999])
    base = torch.zeros((3, 1, 3000), device=DEV)
    one = tk.indexer_scores(*args[:5], out=base.clone())
    for _ in range(20):
        assert torch.equal(tk.indexer_scores(*args[:5], out=base.clone()), one)


def test_example_step():
    """The example's decode step against its own plain form: the selection may
    differ where scores are within rounding of the cutoff, a few entries of
    2 x 10^-3 of the weight each."""
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import sparse_step as ex

    torch.manual_seed(3)
    cache, f, token = ex.make(5, 900)
    got = ex.step(cache, f, *token, 128)
    want = ex.step_plain(cache, f, *token, 128)
    # two roundings of bfloat16 results and one of its weights, then a swapped entry
    assert (got - want).float().norm() <= (3 * 2.0 ** -8 + 0.02) * want.float().norm()


# ---- refusals that need tensors on the GPU -----------------------------------------------------------


def test_refusals():
    f = tk.rotary_frequencies(8, device=DEV)
    x = torch.zeros((2, 2, 8), device=DEV)
    pos = _ints([0, 1])
    for bad in (dict(x=x.double()), dict(positions=pos.float()), dict(positions=pos[:1]), dict(frequencies=f.float()),
                dict(layout="other"), dict(out=x[:1]), dict(out=x.half()), dict(scale=math.nan), dict(slots=pos),
                dict(slots=pos, out=x), dict(slots=pos.long(), out=x[None]), dict(out=x[:1].expand(2, 2, 8)),
                dict(x=x.transpose(1, 2)), dict(x=torch.zeros((3, 2, 8), device=DEV)[:2])):
        kw = dict(x=x, positions=pos, frequencies=f)
        kw.update(bad)
        if bad.keys() == {"x"} and bad["x"].shape == x.shape and bad["x"].is_contiguous() and bad["x"].dtype == FP32:
            base = bad["x"]._base  # an out that overlaps x without being it
            kw["out"] = base[1:]
        with pytest.raises(ValueError):
            tk.rotary(**kw)
    with pytest.raises(tk.TopkError):
        tk.rotary(x, pos, f, offset=1)
    q, w, keys, n, table, _ = _scores_case(2, 1, 8, 64, 64, 16, BF16, [64, 3])
    for bad in (dict(q=q.float()), dict(keys=keys.half()), dict(keys=keys[..., :32]), dict(weights=w.half()),
                dict(weights=w[:1]), dict(lengths=n.long()), dict(page_table=table[:1]), dict(page_table=table.long()),
                dict(key_scales=torch.ones(3, device=DEV)), dict(width=65), dict(out=torch.zeros((2, 1, 65), device=DEV)),
                dict(out=torch.zeros((2, 2, 64), device=DEV)), dict(out=torch.zeros((1, 1, 64), device=DEV).expand(2, 1, 64)),
                dict(page_table=table.cpu())):
        kw = dict(q=q, weights=w, keys=keys, lengths=n, page_table=table)
        kw.update(bad)
        with pytest.raises(ValueError):
            tk.indexer_scores(**kw)
    odd = torch.zeros((keys.shape[0], 16, 68), dtype=BF16, device=DEV)[..., 4:]
    with pytest.raises(tk.TopkError):  # entries that do not start on 16 bytes
        tk.indexer_scores(q, w, odd, n, table)
    with pytest.raises(tk.TopkError):
        tk.indexer_scores(q.repeat(1, 1, 17, 1), w.repeat(1, 1, 17), keys, n, table)  # 136 heads
    q, k, v, idx, table = _attention_case(2, 1, 4, 2, 64, 64, 10, 50, 16, BF16)
    slopes, qpos = torch.zeros(4, device=DEV), _ints([[49], [49]])
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(v=v[:, :8]), dict(q=q[:, :, :3]), dict(indices=idx.long()),
                dict(indices=idx[..., :1].expand(2, 1, 10)), dict(page_table=table[:1]), dict(page_table=None, first=qpos),
                dict(slopes=slopes), dict(slopes=slopes[:3], query_positions=qpos), dict(query_positions=qpos.view(-1)),
                dict(scale=math.inf), dict(softcap=-1.0), dict(softcap=math.nan), dict(out=q.half()), dict(out=q)):
        kw = dict(q=q, k=k, v=v, indices=idx, page_table=table)
        kw.update(bad)
        with pytest.raises(ValueError):
            tk.sparse_attention(**kw)
    with pytest.raises(tk.TopkError):
        wide = torch.zeros((2, 1, 4, 264), dtype=BF16, device=DEV)
        tk.sparse_attention(wide, torch.zeros((4, 16, 2, 264), dtype=BF16, device=DEV), v[:4], idx, table)
