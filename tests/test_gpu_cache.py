"""The operators of a paged cache in 8 bits on the GPU against their formulas in 64 bits (``cache_reference``)."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import cache_reference as C  # noqa: E402
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


def _codes(shape, seed):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * 110.0).clamp(-448.0, 448.0).to(E4M3)


def _scales(shape, seed, low=-9, high=-5):
    return torch.exp2(torch.randint(low, high, shape, generator=_gen(seed), device=DEV).float())


def _sequences(lengths, page_size, pages, seed, spare=0, start=None):
    """(slots, positions) of sequences one behind the other that go on from some place, `spare` idle tokens behind."""
    g = np.random.default_rng(seed)
    order, slots, positions = list(g.permutation(pages)), [], []
    for n in lengths:
        at = int(g.integers(0, 3 * page_size)) if start is None else start
        where = np.arange(at, at + n)
        mine = {p: order.pop() for p in sorted(set(where // page_size))}
        slots += [int(mine[w // page_size]) * page_size + int(w % page_size) for w in where]
        positions += where.tolist()
    return _ints(slots + [-1] * spare), _ints(positions + [0] * spare)


# ---- append: caches in 8 bits ------------------------------------------------------------------------

APPEND = [
    # lengths, H, D, Dv, rotated, offset, layout, page_size, blocks, dtype
    ([1], 1, 64, 64, 64, 0, "half", 64, 1, BF16),
    ([1] * 33, 4, 128, 128, 64, 0, "half", 64, 1, BF16),
    ([200, 1, 63, 64, 65], 3, 128, 64, 128, 0, "half", 64, 1, FP16),
    ([100, 30], 5, 112, 80, 48, 64, "interleaved", 48, 3, FP32),
    ([300], 1, 128, 0, 64, 0, "half", 64, 64, BF16),
    ([17, 3, 50], 2, 96, 40, 0, 0, "half", 17, 1, BF16),  # not rotated
    ([40, 9], 2, 20, 7, 6, 5, "half", 12, 2, BF16),  # nothing aligned
    ([40, 9], 3, 33, 18, 32, 1, "interleaved", 10, 5, FP16),
    ([700], 2, 64, 64, 32, 32, "interleaved", 512, 1, FP32),  # a block of several shares
    ([3], 2, 1022, 1024, 1022, 0, "half", 4, 2, BF16),  # more items than threads
    ([2000, 1111, 1], 9, 64, 64, 64, 0, "half", 64, 4, BF16),  # several heads a thread
    ([5, 6], 33, 16, 16, 16, 0, "interleaved", 1, 1, FP32),
]


def _case(lengths, H, D, Dv, rotated, page_size, blocks, dtype, seed=0, spare=0, start=None):
    pages = sum(-(-n // page_size) + 1 for n in lengths) + 2
    slots, positions = _sequences(lengths, page_size, pages, seed, spare, start)
    T = slots.numel()
    grow = torch.exp2(torch.randint(-3, 4, (H, 1), generator=_gen(seed + 9), device=DEV).float())
    c = dict(k=(_randn((T, H, D), seed + 1) * grow).to(dtype), v=(_randn((T, H, Dv), seed + 2) * grow).to(dtype) if Dv else None,
             slots=slots, positions=positions, f=tk.rotary_frequencies(rotated, device=DEV) if rotated else None,
             k_cache=_codes((pages, page_size, H, D), seed + 3), k_scales=_scales((pages, blocks, H), seed + 4),
             v_cache=None, v_scales=None)
    if Dv:
        c["v_cache"], c["v_scales"] = _codes((pages, page_size, H, Dv), seed + 5), _scales((pages, blocks, H), seed + 6)
    return c


def _append(c, **kw):
    tk.cache_append(c["k"], c["v"], c["positions"], c["f"], c["k_cache"], c["v_cache"], c["slots"],
                    k_scales=c["k_scales"], v_scales=c["v_scales"], **kw)


def _want(c, layout="half", offset=0, scale=1.0):
    """[(name, cache, bound, scales)] that the call leaves."""
    got = []
    for side in ("k", "v"):
        cache, scales = c[side + "_cache"], c[side + "_scales"]
        if cache is None:
            continue
        block = cache.shape[1] // scales.shape[1] if scales is not None else 1
        f = c["f"] if side == "k" else None
        got.append((side, *C.append(c[side], c["positions"], f, cache, scales, c["slots"], block, layout, offset, scale)))
    return got


def _check(c, want):
    for side, cache, bound, scales in want:
        if scales is not None:
            assert np.array_equal(R.np64(c[side + "_scales"]), scales, equal_nan=True), f"{side} scales"
        R.assert_near(c[side + "_cache"].float(), cache, bound, side)


@pytest.mark.parametrize("lengths,H,D,Dv,rotated,offset,layout,page_size,blocks,dtype", APPEND)
def test_append(lengths, H, D, Dv, rotated, offset, layout, page_size, blocks, dtype):
    """Tokens, scales, entries rounded again and everything that has to stay as it was, bit for bit; then the same
    call once more, which changes nothing."""
    c = _case(lengths, H, D, Dv, rotated, page_size, blocks, dtype, spare=3)
    want = _want(c, layout, offset, 1.25)
    _append(c, layout=layout, offset=offset, scale=1.25)
    _check(c, want)
    before = [c[n].clone().view(torch.uint8) if c[n] is not None else None for n in ("k_cache", "v_cache")]
    c["positions"] = c["positions"].long()
    _append(c, layout=layout, offset=offset, scale=1.25)
    for n, b in zip(("k_cache", "v_cache"), before):
        assert b is None or torch.equal(c[n].view(torch.uint8), b)


def test_append_token_by_token():
    """A sequence in chunks of any size: every state is what the formula says of the one before."""
    H, D, ps, blocks = 3, 64, 32, 2
    c = _case([70], H, D, D, D, ps, blocks, BF16, seed=3, start=0)
    c["k_scales"].fill_(math.nan), c["v_scales"].fill_(math.nan)  # of blocks that begin: not looked at
    whole, at = dict(c), 0
    for n in (1, 1, 5, 9, 1, 15, 16, 2, 20):
        for name in ("k", "v", "slots", "positions"):
            c[name] = whole[name][at:at + n].contiguous()
        want = _want(c)
        _append(c)
        _check(c, want)
        at += n
    assert at == 70


def test_append_what_is_not_finite():
    """NaN and infinities become NaN and do not count for the scale; zeros get the least one; numbers near both
    ends of the type's range."""
    H, D, ps = 6, 32, 8
    c = _case([8, 8], H, D, D, D, ps, 1, BF16, seed=5, start=0)
    c["v"][0, 0, 3], c["v"][1, 0, 4], c["k"][2, 0, 5] = math.nan, math.inf, -math.inf
    for side in ("k", "v"):
        c[side][:, 1] = 0.0
        c[side][:, 2] *= 1e36
        c[side][:, 3] *= 1e-38
        c[side][8:, 4] = math.nan
    want = _want(c)
    _append(c)
    _check(c, want)
    assert (c["v_scales"][:, 0, 1] == 2.0 ** -126).sum() == 2
    assert torch.isnan(c["v_cache"].float()).sum() == 2 + 8 * D


def test_append_scale_of_zero():
    """A block whose scale is 0 holds nothing, wherever the first token goes."""
    c = _case([5], 2, 64, 64, 64, 16, 1, BF16, seed=6, start=7)
    c["k_scales"].zero_(), c["v_scales"].zero_()
    c["k_cache"].view(torch.uint8).fill_(0x55), c["v_cache"].view(torch.uint8).fill_(0x55)
    want = _want(c)
    _append(c)
    _check(c, want)


def test_append_places_behind_count_as_empty():
    """A block written again from its middle: the entries behind stay as they are, whatever the scale becomes."""
    c = _case([4], 2, 64, 64, 64, 16, 1, FP16, seed=7, start=6)
    c["k"], c["v"] = c["k"] * 64.0, c["v"] * 64.0
    behind = [c[n].clone() for n in ("k_cache", "v_cache")]
    want = _want(c)
    _append(c)
    _check(c, want)
    page = int(c["slots"][0]) // 16
    for n, b in zip(("k_cache", "v_cache"), behind):
        assert torch.equal(c[n][page, 10:].view(torch.uint8), b[page, 10:].view(torch.uint8))
        assert not torch.equal(c[n][page, :6].view(torch.uint8), b[page, :6].view(torch.uint8))


def test_append_any_scale_before():
    """Scales that are not powers of two, as another quantiser leaves them."""
    c = _case([1] * 40, 4, 128, 64, 64, 32, 2, BF16, seed=8)
    for n in ("k_scales", "v_scales"):
        c[n] *= torch.rand(c[n].shape, generator=_gen(11), device=DEV) + 0.5
    names = ("k_scales", "v_scales")
    old = {n: R.np64(c[n]) for n in names}
    want = _want(c)
    _append(c)
    for side, cache, bound, scales in want:
        assert np.array_equal(R.np64(c[side + "_scales"]), scales)
        # an entry's ratio is rounded, so that one on a border may go either way: a step, where the scale grew
        grown = np.repeat(scales != old[side + "_scales"], 16, axis=1)[..., None]
        R.assert_near(c[side + "_cache"].float(), cache, bound + grown * np.maximum(np.abs(cache) * 2.0 ** -3, 2.0 ** -9), side)


def test_append_slots_that_are_not_in_the_cache():
    """Slots past the cache, negative ones between tokens, none at all, no page, no token."""
    c = _case([6], 2, 64, 64, 64, 8, 8, BF16, seed=9)
    c["slots"] = _ints([3, -1, 8 * c["k_cache"].shape[0], 0, -2 ** 31, 2 ** 31 - 1])
    want = _want(c)
    _append(c)
    _check(c, want)
    c["slots"].fill_(-1)
    before = [c[n].clone() for n in ("k_cache", "v_cache", "k_scales", "v_scales")]
    _append(c)
    for n, b in zip(("k_cache", "v_cache", "k_scales", "v_scales"), before):
        assert torch.equal(c[n].float(), b.float())
    for n in ("k", "v", "slots", "positions"):
        c[n] = c[n][:0]
    _append(c)
    c = _case([6], 2, 64, 64, 64, 8, 8, BF16, seed=9)
    for n in ("k_cache", "v_cache", "k_scales", "v_scales"):
        c[n] = c[n][:0]
    _append(c)


def test_append_strides():
    """Keys and values out of one joint tensor, caches that are parts of one, tokens and heads in any order."""
    H, D, ps, pages = 3, 64, 16, 9
    c = _case([40, 3], H, D, D, D, ps, 2, BF16, seed=10)
    T = c["slots"].numel()
    joint = torch.empty((H, T, 2 * D + 8), dtype=BF16, device=DEV).transpose(0, 1)
    joint[..., :D], joint[..., D + 8:] = c["k"], c["v"]
    for shape, parts in (((pages, 2, ps, H, D), lambda t: (t[:, 0], t[:, 1])),
                         ((pages, ps, H, 2 * D), lambda t: (t[..., :D], t[..., D:])),
                         ((pages, H, ps, 2 * D + 4), lambda t: (t[..., :D].transpose(1, 2), t[..., D + 4:].transpose(1, 2)))):
        both = _codes(shape, 1)
        before = both.clone()
        c["k_cache"], c["v_cache"] = parts(both)
        c["k_scales"], c["v_scales"] = _scales((pages, 2, H), 2), _scales((pages, 2, H), 3)
        want = _want(c)
        c["k"], c["v"] = joint[..., :D], joint[..., D + 8:]
        _append(c)
        _check(c, want)
        if shape[-1] > 2 * D:
            assert torch.equal(both[..., D:D + 4].view(torch.uint8), before[..., D:D + 4].view(torch.uint8))


@pytest.mark.parametrize("dtype,H,D,Dv,rotated,offset,layout", [
    (BF16, 8, 128, 128, 128, 0, "half"), (FP16, 3, 80, 33, 32, 8, "interleaved"), (FP32, 5, 96, 64, 48, 0, "half"),
    (FP16, 2, 20, 18, 6, 5, "half"), (BF16, 1, 64, 0, 0, 0, "half")])
def test_append_16_and_32_bits(dtype, H, D, Dv, rotated, offset, layout):
    """Caches of the inputs' type, slots in any order."""
    T, ps, pages = 300, 16, 21
    f = tk.rotary_frequencies(rotated, device=DEV) if rotated else None
    c = dict(k=_randn((T, H, D), 1, dtype), v=_randn((T, H, Dv), 2, dtype) if Dv else None, f=f, k_scales=None, v_scales=None,
             positions=torch.randint(-5, 1 << 20, (T,), generator=_gen(3), device=DEV).to(torch.int32),
             slots=torch.randperm(pages * ps, generator=_gen(4), device=DEV)[:T].to(torch.int32),
             k_cache=_randn((pages, ps, H, D), 5, dtype), v_cache=_randn((pages, ps, H, Dv), 6, dtype) if Dv else None)
    c["slots"][5::7] = -1
    want = _want(c, layout, offset, 0.75)
    _append(c, layout=layout, offset=offset, scale=0.75)
    _check(c, want)


def test_append_far_slots():
    """Slots and tokens whose elements lie past 2^32."""
    pages, ps, H, D = 70, 64, 1, 128
    wide = torch.zeros(2 ** 32 + 2 ** 29, dtype=torch.uint8, device=DEV).view(E4M3)
    cache = wide.as_strided((pages, ps, H, D), (2 ** 26 - 2 ** 18, 2 ** 19 + 16, D, 1))
    scales = torch.ones((pages, 1, H), device=DEV)
    slots, positions = _ints([69 * 64 + 62, 69 * 64 + 63, 5]), _ints([7, 8, 9])
    k = _randn((3, H, D), 1, BF16)
    f = tk.rotary_frequencies(D, device=DEV)
    want, bound, units = C.append(k, positions, f, cache[[0, 69]].contiguous(), scales[[0, 69]],
                                  _ints([64 + 62, 64 + 63, 5]), 64)
    tk.cache_append(k, None, positions, f, cache, None, slots, k_scales=scales)
    R.assert_near(cache[[0, 69]].float(), want, bound)
    assert np.array_equal(R.np64(scales[[0, 69]]), units) and (scales[1:69] == 1.0).all()


def test_append_in_a_graph_and_on_a_stream():
    """Captured once, replayed on tokens and slots that changed since; on a stream of the caller's."""
    c = _case([1] * 20, 4, 128, 128, 64, 64, 1, BF16, seed=12)
    _append(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _append(c)
    for seed in range(3):
        c["k"].copy_(_randn(c["k"].shape, 20 + seed, BF16, 4.0 ** seed)), c["v"].copy_(_randn(c["v"].shape, 30 + seed, BF16, 0.3))
        c["slots"].copy_(torch.where(c["slots"] % 64 < 63, c["slots"] + 1, c["slots"]))
        c["positions"].add_(1)
        want = _want(c)
        graph.replay()
        _check(c, want)
    side = torch.cuda.Stream()
    c["k"].mul_(32.0)
    want = _want(c)
    torch.cuda.synchronize()
    _append(c, stream=side)
    side.synchronize()
    _check(c, want)
