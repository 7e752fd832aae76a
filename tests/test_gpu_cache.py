"""The operators of a paged cache in 8 bits on the GPU against their formulas in 64 bits (``cache_reference``)."""

import ctypes
import math
import os
import subprocess
import sys

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


# ---- attention over a cache in 8 bits ----------------------------------------------------------------


def _attend(B, T, Hq, Hkv, D, Dv, K, S, ps, blocks, dtype, seed=0, shared=False, spread=1.0, **more):
    """The arguments of a call on ragged sequences in a pool whose unread parts are NaN, scales among them."""
    g, pages = _gen(seed), -(-S // ps)
    pool = B * pages + 3
    table = torch.randperm(pool, generator=g, device=DEV)[:B * pages].to(torch.int32).view(B, pages)
    k, ks = _codes((pool, ps, Hkv, D), seed + 1), torch.exp2(torch.rand((pool, blocks, Hkv), generator=g, device=DEV) * 2 - 8.5)
    v, vs = _codes((pool, ps, Hkv, Dv), seed + 2), torch.exp2(torch.rand((pool, blocks, Hkv), generator=g, device=DEV) * 2 - 8.5)
    if shared:
        v, vs = k[..., :Dv], ks
    last = torch.randint(S // 2, S, (B, 1), generator=g, device=DEV)
    qpos = (last - T + 1 + torch.arange(T, device=DEV)).clamp(min=0).to(torch.int32)
    idx = torch.stack([torch.stack([torch.randperm(S, generator=g, device=DEV)[:K] if K <= S else
                                    torch.randint(0, S, (K,), generator=g, device=DEV) for _ in range(T)]) for _ in range(B)])
    idx = torch.where(torch.rand(idx.shape, generator=g, device=DEV) < 0.05, -1, idx).to(torch.int32)
    # entries that no row sees, and scales of blocks without one that is seen, are NaN
    used = torch.zeros((pool, ps), dtype=torch.bool, device=DEV)
    for b in range(B):
        seen = idx[b][(idx[b] >= 0) & (idx[b] <= qpos[b][:, None])].long()
        used[table[b].long()[seen // ps], seen % ps] = True
    free = ~used.view(pool, blocks, -1).any(-1)
    k.view(torch.uint8)[~used] = 0x7f
    ks[free] = math.nan
    if not shared:
        v.view(torch.uint8)[~used] = 0x7f
        vs[free] = math.nan
    q = _randn((B, T, Hq, D), seed + 3, dtype, 1.5 * spread)
    return dict(q=q, k=k, v=v, indices=idx.contiguous(), page_table=table, k_scales=ks, v_scales=vs, query_positions=qpos,
                scale=D ** -0.5, **more)


def _attention_check(c, what=""):
    out, lse = tk.sparse_attention(**c, return_lse=True)
    clean = {n: torch.nan_to_num(c[n].float(), nan=0.0) for n in ("k_scales", "v_scales")}
    k, v = (torch.where(torch.isnan(c[n].float()), 0.0, c[n].float()).to(E4M3) for n in ("k", "v"))
    want = C.attention(c["q"], k, v, clean["k_scales"], clean["v_scales"], c["indices"], c.get("page_table"),
                       c.get("query_positions"), c["scale"], c.get("softcap", 0.0), c.get("slopes"), c.get("first"))
    R.assert_near(lse, want[2], want[3], what + " lse")
    R.assert_near(out, want[0], want[1], what + " out")
    return out, lse


ATTEND = [
    # B, T, Hq, Hkv, D, Dv, K, S, page_size, blocks, dtype
    (1, 1, 8, 1, 128, 128, 128, 300, 64, 1, BF16),
    (1, 1, 1, 1, 64, 64, 1, 5, 16, 1, BF16),
    (2, 1, 32, 4, 128, 128, 512, 1000, 64, 4, BF16),
    (2, 1, 32, 4, 128, 128, 512, 1000, 64, 4, FP16),
    (3, 2, 15, 5, 96, 64, 129, 400, 17, 17, FP16),
    (3, 2, 14, 2, 80, 144, 127, 400, 51, 3, BF16),
    (1, 3, 24, 2, 16, 16, 300, 400, 1, 1, BF16),  # 12 heads
    (1, 3, 32, 2, 128, 128, 300, 400, 64, 1, FP16),
    (2, 1, 20, 1, 256, 192, 200, 333, 48, 6, BF16),
    (2, 1, 64, 2, 192, 256, 260, 333, 48, 6, FP16),
    (1, 2, 64, 1, 256, 256, 270, 500, 64, 64, BF16),
    (1, 2, 50, 1, 128, 80, 270, 500, 64, 2, FP16),  # two tiles of heads in fp16
    (1, 1, 150, 1, 64, 64, 200, 500, 64, 1, BF16),  # three tiles of heads
    (1, 1, 8, 1, 128, 128, 2048, 5000, 64, 1, BF16),  # a cluster of eight
    (1, 1, 64, 1, 128, 128, 1000, 5000, 64, 1, BF16),
    (5, 1, 40, 1, 64, 240, 700, 900, 256, 2, FP16),
    (2, 2, 4, 4, 32, 32, 6, 4, 4, 2, BF16),  # more entries than positions: listed twice
    (170, 2, 8, 1, 64, 64, 130, 140, 16, 1, BF16),  # more works than places
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,Dv,K,S,ps,blocks,dtype", ATTEND)
def test_attention(B, T, Hq, Hkv, D, Dv, K, S, ps, blocks, dtype):
    _attention_check(_attend(B, T, Hq, Hkv, D, Dv, K, S, ps, blocks, dtype, seed=K))


@pytest.mark.parametrize("heads,D,Dv,dtype", [(8, 128, 128, BF16), (64, 256, 192, BF16), (16, 256, 256, FP16), (128, 128, 64, BF16),
                                              (30, 144, 48, FP16)])
def test_attention_shared_entries(heads, D, Dv, dtype):
    """Values that are the first elements of the keys."""
    _attention_check(_attend(2, 3, heads, 1, D, Dv, 333, 600, 64, 64, dtype, seed=heads, shared=True))


@pytest.mark.parametrize("heads,dtype", [(8, BF16), (16, FP16), (40, BF16)])
@pytest.mark.parametrize("cap", [0.0, 1e-3, 5.0, 30.0])
@pytest.mark.parametrize("bias", [False, True])
def test_attention_cap_bias_documents(heads, dtype, cap, bias):
    c = _attend(2, 2, heads, 1, 64, 64, 300, 500, 32, 2, dtype, seed=5, softcap=cap, spread=3.0)
    if bias:
        c["slopes"] = _randn((heads,), 6, FP32, 0.05)
    c["first"] = (c["query_positions"] * 0.3).to(torch.int32)
    c["first"][0, 1] = 2 ** 31 - 1  # a row that sees nothing
    c["first"][1, 0] = -5
    out, lse = _attention_check(c)
    assert (out[0, 1] == 0).all() and torch.isneginf(lse[0, 1]).all()


def test_attention_that_sees_nothing():
    """No entry, no index, no page, pages outside the cache and the table."""
    c = _attend(2, 1, 8, 2, 64, 64, 40, 100, 16, 1, BF16)
    for change in (dict(indices=torch.full_like(c["indices"], -1)), dict(indices=c["indices"][..., :0].contiguous()),
                   dict(page_table=torch.full_like(c["page_table"], -1)), dict(page_table=torch.full_like(c["page_table"], 2 ** 31 - 1)),
                   dict(page_table=c["page_table"][:, :0]), dict(query_positions=torch.full_like(c["query_positions"], -1)),
                   dict(k=c["k"][:0], v=c["v"][:0], k_scales=c["k_scales"][:0], v_scales=c["v_scales"][:0])):
        out, lse = tk.sparse_attention(**{**c, **change}, return_lse=True)
        assert (out == 0).all() and torch.isneginf(lse).all(), change.keys()
    assert tk.sparse_attention(**{**c, "q": c["q"][:0], "indices": c["indices"][:0], "page_table": c["page_table"][:0],
                                  "query_positions": c["query_positions"][:0]}).shape == (0, 1, 8, 64)


def test_attention_slots_and_strides():
    """Slots instead of positions; caches that are parts of one, queries that are not aligned, a shared page table."""
    H, D, ps, pages, K = 2, 64, 16, 20, 200
    both = _codes((pages, 2, ps, H, D), 1)
    ks, vs = _scales((pages, 4, H), 2), _scales((pages, 4, H), 3)
    idx = torch.randint(-1, pages * ps, (2, 3, K), generator=_gen(4), device=DEV).to(torch.int32)
    joint = _randn((2, 3, 8 * D + 9), 5, FP16)
    q = joint[..., 3:3 + 8 * D].unflatten(-1, (8, D))
    c = dict(q=q, k=both[:, 0], v=both[:, 1], indices=idx, k_scales=ks, v_scales=vs, scale=0.2)
    one = _attention_check(c, "slots")
    table = torch.arange(pages, dtype=torch.int32, device=DEV).expand(2, pages)
    two = _attention_check({**c, "page_table": table}, "shared table")
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    out = torch.empty((2, 3, 8, D), dtype=FP16, device=DEV)
    assert tk.sparse_attention(**c, out=out) is out and torch.equal(out, one[0])


@pytest.mark.parametrize("heads,dtype", [(8, BF16), (8, FP16), (16, BF16), (32, FP16), (64, BF16)])
def test_attention_whose_logits_grow(heads, dtype):
    """Every tile's logits above those of the one before, by little and by much: the references move each time. Then
    one entry far above a flat rest, which the smallest weights carry."""
    D, K, ps = 64, 900, 16
    c = _attend(1, 1, heads, 1, D, D, K, K, ps, 1, dtype, seed=7)
    c["k"], c["v"] = _codes(c["k"].shape, 1), _codes(c["v"].shape, 2)
    c["k_scales"], c["v_scales"] = _scales(c["k_scales"].shape, 3), _scales(c["v_scales"].shape, 4)
    c["indices"] = torch.arange(K, dtype=torch.int32, device=DEV).view(1, 1, K)
    c["query_positions"] = _ints([[K]])
    c["slopes"] = torch.linspace(0.0005, 0.5, heads, device=DEV)
    _attention_check(c, "growing")
    c["slopes"] = -c["slopes"]
    _attention_check(c, "falling")
    del c["slopes"]
    for at in (0, 500, K - 1):
        flat = c["k"].clone()
        flat[...] = 0.0
        page, place = int(c["page_table"][0, at // ps]), at % ps
        c["q"][..., 0] = 3.0
        flat[page, place, 0, 0] = 448.0
        for logit in (5.0, 9.0, 12.0):
            units = torch.full_like(c["k_scales"], logit / (448.0 * 3.0 * c["scale"]))
            _attention_check({**c, "k": flat, "k_scales": units}, f"one above the rest by {logit}")


@pytest.mark.parametrize("heads,Dv,dtype", [(8, 256, BF16), (8, 64, FP16), (16, 144, BF16), (16, 256, FP16), (32, 256, BF16),
                                            (32, 128, FP16), (64, 256, BF16), (64, 128, BF16)])
def test_attention_some_heads_references_move(heads, Dv, dtype):
    """Heads of very different logits: in each tile a few references move, by a little or far, over one or two blocks
    of values, in several rows a CTA."""
    c = _attend(3, 2, heads, 1, 128, Dv, 700, 900, 64, 4, dtype, seed=heads + Dv)
    c["q"] = c["q"] * torch.exp2((torch.arange(heads, device=DEV) * 5 % 7 - 3).float())[:, None].to(dtype)
    _attention_check(c)


@pytest.mark.parametrize("heads,dtype", [(8, BF16), (16, FP16), (64, BF16)])
@pytest.mark.parametrize("order", [1, -1])
def test_attention_near_entries_behind_far_ones(heads, dtype, order):
    """Two entries near the query, and a tile (or several) thousands of positions away, before them or behind: what the
    far ones leave of the near ones' logits is as exact as without them."""
    D, ps, now = 64, 64, 9000
    c = _attend(1, 1, heads, 1, D, D, 2, now + 1, ps, 1, dtype, seed=21)
    c["k"], c["v"] = _codes(c["k"].shape, 1), _codes(c["v"].shape, 2)
    c["k_scales"], c["v_scales"] = _scales(c["k_scales"].shape, 3), _scales(c["v_scales"].shape, 4)
    c["query_positions"], c["slopes"] = _ints([[now]]), torch.full((heads,), 1.0, device=DEV)
    near = [now - 1, now]
    c["indices"] = _ints(near).view(1, 1, 2)
    _attention_check(c, "alone")
    for far in (128, 300):
        idx = _ints((list(range(far)) + near)[::order]).view(1, 1, far + 2)
        # the far entries' weights are 0: the bound is that of two entries
        want = C.attention(c["q"], c["k"], c["v"], c["k_scales"], c["v_scales"], c["indices"], c["page_table"], c["query_positions"],
                           c["scale"], 0.0, c["slopes"])
        out, lse = tk.sparse_attention(**{**c, "indices": idx}, return_lse=True)
        R.assert_near(lse, want[2], want[3], f"lse, {far} far")
        R.assert_near(out, want[0], want[1], f"out, {far} far")


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_attention_scales_far_apart(dtype):
    """Scales of 0, of the least size, and of sizes 2^40 apart, those of the keys and of the values."""
    c = _attend(2, 1, 8, 1, 64, 64, 400, 400, 16, 2, dtype, seed=8)
    c["k"], c["v"] = _codes(c["k"].shape, 1), _codes(c["v"].shape, 2)
    base = _scales(c["k_scales"].shape, 3)
    for far in (0.0, 2.0 ** -126, 2.0 ** -40, 2.0 ** 30):
        odd = base.clone()
        odd[::3] = far
        c["k_scales"], c["v_scales"] = base, odd
        _attention_check(c, f"values {far}")
        c["k_scales"], c["v_scales"] = (odd if far < 1.0 else base), base
        _attention_check(c, f"keys {far}")
    c["v_scales"] = torch.zeros_like(base)
    assert (_attention_check(c, "no values")[0] == 0).all()


def test_attention_what_is_not_finite():
    """A query's NaN or infinity makes NaN of its head, an entry's NaN of what it enters."""
    c = _attend(2, 1, 16, 2, 64, 64, 300, 400, 16, 2, BF16, seed=9)
    c["k"], c["v"] = _codes(c["k"].shape, 1), _codes(c["v"].shape, 2)
    c["k_scales"], c["v_scales"] = _scales(c["k_scales"].shape, 3), _scales(c["v_scales"].shape, 4)
    good, lse = _attention_check(c)
    q = c["q"].clone()
    q[0, 0, 3, 5], q[1, 0, 9, 0] = math.nan, math.inf
    out, got = tk.sparse_attention(**{**c, "q": q}, return_lse=True)
    for b, h in ((0, 3), (1, 9)):
        assert torch.isnan(out[b, 0, h]).all() and torch.isnan(got[b, 0, h])
        out[b, 0, h], got[b, 0, h] = good[b, 0, h], lse[b, 0, h]
    assert torch.equal(out, good) and torch.equal(got, lse)
    seen = c["indices"][0, 0][(c["indices"][0, 0] >= 0) & (c["indices"][0, 0] <= c["query_positions"][0, 0])][-1].item()
    page, place = int(c["page_table"][0, seen // 16]), seen % 16
    v = c["v"].clone()
    v[page, place, 1, 7] = math.nan
    out, got = tk.sparse_attention(**{**c, "v": v}, return_lse=True)
    assert torch.isnan(out[0, 0, 8:, 7]).all() and torch.isnan(out).sum() == 8 and torch.equal(got, lse)
    k = c["k"].clone()
    k[page, place, 0, 1] = math.nan
    out, got = tk.sparse_attention(**{**c, "k": k}, return_lse=True)
    assert torch.isnan(out[0, 0, :8]).all() and torch.isnan(got[0, 0, :8]).all()
    assert torch.equal(out[0, 0, 8:], good[0, 0, 8:]) and torch.equal(out[1], good[1])


def test_attention_far_entries():
    """Entries whose offsets pass 2^32."""
    pages, ps, H, D = 70, 64, 1, 128
    wide = torch.zeros(2 ** 32 + 2 ** 29, dtype=torch.uint8, device=DEV).view(E4M3)
    k = wide.as_strided((pages, ps, H, D), (2 ** 26 - 2 ** 18, 2 ** 19 + 16, D, 1))
    idx = torch.cat([torch.arange(65 * 64, 70 * 64), torch.arange(0, 70)]).to(torch.int32).to(DEV).view(1, 1, -1)
    k[65:], k[:2] = _codes((5, ps, H, D), 1), _codes((2, ps, H, D), 2)
    scales = _scales((pages, 1, H), 3)
    c = dict(q=_randn((1, 1, 6, D), 4, BF16), k=k, v=k[..., :64], indices=idx, k_scales=scales, v_scales=scales, scale=0.1)
    got = tk.sparse_attention(**c, return_lse=True)
    near = torch.cat([idx[..., :320] - 65 * 64, idx[..., 320:] + 5 * 64], dim=-1).to(torch.int32).contiguous()
    few = torch.cat([k[65:], k[:2]]).contiguous()
    some = torch.cat([scales[65:], scales[:2]]).contiguous()
    want = tk.sparse_attention(c["q"], few, few[..., :64], near, k_scales=some, v_scales=some, scale=0.1, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_in_a_graph_and_on_streams():
    """Captured and replayed on other indices, and side by side with itself and with the 16-bit attention on two streams."""
    c = _attend(20, 1, 32, 4, 128, 128, 600, 700, 64, 1, BF16, seed=11)
    c["k"], c["v"] = _codes(c["k"].shape, 1), _codes(c["v"].shape, 2)
    c["k_scales"], c["v_scales"] = _scales(c["k_scales"].shape, 3), _scales(c["v_scales"].shape, 4)
    out = torch.empty((20, 1, 32, 128), dtype=BF16, device=DEV)
    tk.sparse_attention(**c, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tk.sparse_attention(**c, out=out)
    for seed in range(3):
        c["indices"].copy_(torch.randint(-1, 700, c["indices"].shape, generator=_gen(seed), device=DEV))
        c["q"].copy_(_randn(c["q"].shape, seed, BF16))
        graph.replay()
        assert torch.equal(out, tk.sparse_attention(**c))
    wide = _attend(3, 1, 64, 1, 256, 192, 900, 1000, 64, 1, BF16, seed=12, shared=True)
    k16 = _randn((300, 16, 4, 128), 2, BF16)
    some = torch.randint(-1, 4800, (40, 1, 600), generator=_gen(3), device=DEV).to(torch.int32)
    q16, wide16 = _randn((40, 1, 32, 128), 1, BF16), _randn((40, 1, 256, 128), 1, BF16)
    calls = [lambda: tk.sparse_attention(**c), lambda: tk.sparse_attention(**wide),
             lambda: tk.sparse_attention(q16, k16, k16, some), lambda: tk.sparse_attention(wide16, k16, k16, some)]
    want = [call() for call in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for turn in range(1, len(calls)):
        got = [[], []]
        for _ in range(10):
            for i in range(len(calls)):
                for side, stream in enumerate(streams):
                    with torch.cuda.stream(stream):
                        got[side].append(calls[(i + side * turn) % len(calls)]())
        torch.cuda.synchronize()
        for side in range(2):
            for i, g in enumerate(got[side]):
                assert torch.equal(g, want[(i + side * turn) % len(calls)])


# ---- the whole way -----------------------------------------------------------------------------------


def test_first_calls_of_a_process_are_captured():
    """Nothing has to run eagerly before: a graph of the first calls gives what they give."""
    code = """
import torch, sparse_attention_indexer_fp32_gb300 as tk
def randn(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)
torch.manual_seed(0)
k, v, q = randn(128, 2, 64), randn(128, 2, 64), randn(1, 1, 16, 64)
caches = [torch.zeros((2, 64, 2, 64), device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
scales = [torch.zeros((2, 1, 2), device="cuda") for _ in range(2)]
slots = torch.arange(128, dtype=torch.int32, device="cuda")
listed, freq = slots.view(1, 1, 128).clone(), tk.rotary_frequencies(64, device="cuda")
out = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
def call():
    tk.cache_append(k, v, slots, freq, *caches, slots, k_scales=scales[0], v_scales=scales[1])
    tk.sparse_attention(q, *caches, listed, k_scales=scales[0], v_scales=scales[1], out=out)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = [t.view(torch.uint8).clone() for t in (*caches, *scales, out)]
assert out.abs().max() > 0
call()
torch.cuda.synchronize()
assert all(torch.equal(a, t.view(torch.uint8)) for a, t in zip(got, (*caches, *scales, out)))
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=120,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_step_in_8_bits(dtype):
    """Prompts and then single tokens appended (keys and values; the indexer's keys with a scale each), scores over the
    8-bit keys, the selection and attention over the 8-bit entries: each call on what the one before left."""
    B, Hq, Hkv, D, ps, blocks, H, select = 3, 16, 2, 64, 32, 2, 8, 512
    pages, f = 24, tk.rotary_frequencies(32, device=DEV)
    table = torch.randperm(B * pages, generator=_gen(1), device=DEV).to(torch.int32).view(B, pages)
    caches = [torch.zeros((B * pages, ps, Hkv, D), device=DEV).to(E4M3) for _ in range(2)]
    scales = [torch.zeros((B * pages, blocks, Hkv), device=DEV) for _ in range(2)]
    index_cache = torch.zeros((B * pages, ps, 1, D), device=DEV).to(E4M3)
    index_scales = torch.zeros((B * pages, ps, 1), device=DEV)
    held = [[], [], []]  # what was appended, in 64 bits, by sequence
    at = torch.zeros(B, dtype=torch.int64)
    for step, counts in enumerate(([601, 0, 330], [1, 1, 1], [1, 0, 1], [1, 40, 1])):
        T = sum(counts) + 2  # idle tokens behind the last sequence
        k, v = _randn((T, Hkv, D), 10 + step, dtype, 2.0 ** step), _randn((T, Hkv, D), 20 + step, dtype, 2.0 ** -step)
        ik = _randn((T, 1, D), 30 + step, dtype)
        where = [int(at[b]) + i for b in range(B) for i in range(counts[b])]
        owner = [b for b in range(B) for _ in range(counts[b])]
        slots = _ints([int(table[b, w // ps]) * ps + w % ps for b, w in zip(owner, where)] + [-1, -1])
        positions = _ints(where + [0, 0])
        tk.cache_append(k, v, positions, f, *caches, slots, k_scales=scales[0], v_scales=scales[1])
        tk.cache_append(ik, None, positions, f, index_cache, None, slots, k_scales=index_scales)
        turned = [R.np64(tk.rotary(x.float(), positions, f)) for x in (k, ik)]
        for b in range(B):
            mine = [i for i, o in enumerate(owner) if o == b]
            held[b].append([turned[0][mine], R.np64(v)[mine], turned[1][mine]])
        at += torch.tensor(counts)
    lengths = at.to(torch.int32).to(DEV)
    width = pages * ps
    iq, w = _randn((B, 1, H, D), 2), _randn((B, 1, H), 3)
    scores = tk.indexer_scores((iq * 16.0).to(E4M3), w, index_cache[:, :, 0], lengths[:, None], table, key_scales=index_scales[..., 0],
                               out=torch.zeros((B, 1, width), device=DEV))
    chosen = tk.topk_ragged(scores.view(B, width), lengths, select)
    q = _randn((B, 1, Hq, D), 4, dtype)
    c = dict(q=q, k=caches[0], v=caches[1], indices=chosen[:, None].contiguous(), page_table=table, k_scales=scales[0],
             v_scales=scales[1], query_positions=(lengths - 1)[:, None].contiguous(), scale=D ** -0.5)
    out, lse = _attention_check(c)
    # and against what was appended, before any rounding to 8 bits
    flat = [R.np64(t.float()).reshape(B * pages, blocks, ps // blocks, Hkv, D) * R.np64(s)[:, :, None, :, None] for t, s in zip(caches, scales)]
    index_flat = R.np64(index_cache.float()) * R.np64(index_scales)[..., None]
    for b in range(B):
        parts = [np.concatenate([h[i] for h in held[b]]) for i in range(3)]
        order = np.asarray([int(table[b, p // ps]) * ps + p % ps for p in range(int(at[b]))])
        for got, want, unit in ((flat[0], parts[0], scales[0]), (flat[1], parts[1], scales[1])):
            got = got.reshape(-1, Hkv, D)[order]
            units = np.repeat(R.np64(unit), ps // blocks, axis=1).reshape(-1, Hkv)[order][..., None]
            # rounded once and, where a scale grew, again below the type's normal numbers, for each of three growths
            assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 2.0 ** -18) + 4 * 2.0 ** -10 * units).all()
        assert (np.abs(index_flat.reshape(-1, 1, D)[order] - parts[2]) <= np.abs(parts[2]) * (2.0 ** -4 + 2.0 ** -18)
                + 2.0 ** -10 * R.np64(index_scales).reshape(-1, 1)[order][..., None]).all()
        # the selection is that of the scores of the 8-bit entries
        n, idx = int(at[b]), chosen[b][chosen[b] >= 0].cpu().numpy()
        s = scores[b, 0, :n].cpu().numpy()
        assert len(idx) == min(n, select) and (n <= select or s[idx].min() >= np.delete(s, idx).max())
        # attention on the numbers themselves: the 8-bit entries are within 2^-4 of them
        kk, vv = (p[idx].repeat(Hq // Hkv, axis=1) for p in parts[:2])
        z = np.einsum("hd,nhd->hn", R.np64(q)[b, 0], kk) * D ** -0.5
        p = np.exp(z - z.max(axis=1, keepdims=True))
        want = np.einsum("hn,nhd->hd", p / p.sum(axis=1, keepdims=True), vv)
        assert np.linalg.norm(R.np64(out)[b, 0] - want) < 0.25 * np.linalg.norm(want)


# ---- waits that run out ------------------------------------------------------------------------------


@pytest.fixture(scope="module")
def hurried(tmp_path_factory):
    """The library's calls once more, with waits that give up at once or after 3 us: {limit in ns: {call: its function}}."""
    from sparse_attention_indexer_fp32_gb300 import _step
    from sparse_attention_indexer_fp32_gb300 import build as cuda_build

    units = ["cache_abi.cu", "cache_append.cu", "cache_attention_bf16.cu", "cache_attention_fp16.cu"]
    out = tmp_path_factory.mktemp("hurried_cache")
    jobs = []
    for ns in (0, 3000):
        for u in units:
            jobs.append(subprocess.Popen([cuda_build.nvcc(), *cuda_build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                                          "-I", cuda_build.INCLUDE, f"-DSPARSE_WAIT_LIMIT_NS={ns}", "-c",
                                          os.path.join(cuda_build.CSRC, u), "-o", str(out / f"{ns}_{u}.o")]))
    assert [job.wait() for job in jobs] == [0] * len(jobs)
    calls = {}
    for ns in (0, 3000):
        path = str(out / f"libhurried_cache_{ns}.so")
        subprocess.check_call([cuda_build.nvcc(), *cuda_build.ARCH, "-shared", "-o", path, *(str(out / f"{ns}_{u}.o") for u in units)])
        prototype = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, ctypes.c_void_p)
        call = _step._attention_e4m3
        calls[ns] = {call: prototype(ctypes.cast(getattr(ctypes.CDLL(path), call.name), ctypes.c_void_p).value)}
    return calls


@pytest.mark.parametrize("rows,Hq,Hkv,K,dtype", [(1, 8, 1, 2048, BF16), (3, 16, 4, 700, FP16), (400, 8, 1, 300, BF16),
                                                 (2, 40, 1, 900, BF16), (340, 40, 1, 130, FP16), (340, 64, 1, 400, BF16),
                                                 (330, 12, 1, 200, BF16)])
def test_attention_whose_waits_run_out(hurried, monkeypatch, rows, Hq, Hkv, K, dtype):
    """With waits that run out each number is what it is without, or NaN, and the calls after are right again."""
    D, ps = 64, 16
    q, k, v = _randn((rows, 1, Hq, D), 1, dtype), _codes((200, ps, Hkv, D), 2), _codes((200, ps, Hkv, D), 3)
    ks, vs = _scales((200, 1, Hkv), 4), _scales((200, 1, Hkv), 5)
    idx = torch.randint(-1, 200 * ps, (rows, 1, K), generator=_gen(6), device=DEV).to(torch.int32)

    def call():
        return tk.sparse_attention(q, k, v, idx, k_scales=ks, v_scales=vs, softcap=30.0, return_lse=True)

    want = call()
    for ns in (0, 3000, 0):
        with monkeypatch.context() as patch:
            for entry, fn in hurried[ns].items():
                patch.setattr(entry, "fn", fn)
            got = call()
        torch.cuda.synchronize()
        lost = 0
        for g, w in zip(got, want):
            nan = torch.isnan(g)
            lost += int(nan.sum())
            assert torch.equal(torch.where(nan, w, g), w), f"neither right nor NaN with a limit of {ns} ns"
        assert ns > 0 or lost > 0, "no wait ran out"
        for g, w in zip(call(), want):
            assert torch.equal(g, w), f"the call after one with a limit of {ns} ns"


def test_refusals():
    """What the binding cannot hand on: scales of another shape, caches that overlap, types that do not go together."""
    c = _attend(2, 1, 8, 2, 64, 64, 40, 100, 16, 2, BF16)
    bad = [(dict(v_scales=None), "v_scales"), (dict(k_scales=None), "k_scales"), (dict(k_scales=c["k_scales"][:, :1]), "contiguous"),
           (dict(v_scales=c["v_scales"].sum(1, keepdim=True)), "blocks of k_scales"), (dict(k=c["k"].float()), "float8"),
           (dict(k_scales=None, v_scales=None), "k must be"), (dict(q=c["q"].float()), "q must be"),
           (dict(k_scales=c["k_scales"].double()), "float32")]
    for change, match in bad:
        with pytest.raises(ValueError, match=match):
            tk.sparse_attention(**{**c, **change})
    a = _case([6], 2, 64, 64, 64, 8, 2, BF16)
    both = _codes((4, 8, 2, 100), 1)
    bad = [(dict(k_scales=None), "k_scales"), (dict(v_scales=a["k_scales"]), "its own"), (dict(v=None), "go together"),
           (dict(v_cache=a["v_cache"].float()), "v_cache must be"), (dict(v_cache=a["k_cache"]), "overlap k_cache"),
           (dict(v_cache=a["v_cache"].to(BF16)), "type of k_cache"), (dict(k_cache=both[..., :64], v_cache=both[..., 36:]), "overlap"),
           (dict(v=a["v"].half()), "v must be"), (dict(slots=a["slots"].long()), "slots"), (dict(k=a["k"].double()), "k must be"),
           (dict(f=a["f"].float()), "frequencies"), (dict(positions=None), "positions"),
           (dict(v_scales=a["v_scales"][:, :1].contiguous()), "blocks of k_scales"),
           (dict(k_cache=a["k_cache"][:, :, :, :1].expand(-1, -1, -1, 64)), "unit stride"),
           (dict(k_cache=a["k_cache"][:1].expand(9, -1, -1, -1)), "broadcast")]
    for change, match in bad:
        with pytest.raises(ValueError, match=match):
            _append({**a, **change})
    with pytest.raises(ValueError, match="float8_e4m3fn have scales"):
        _append({**a, "k_cache": a["k_cache"].to(BF16), "v_cache": a["v_cache"].to(BF16)})
    with pytest.raises(tk.TopkError):
        _append(a, offset=2)
    versions = [a[n]._version for n in ("k_cache", "v_scales")]
    _append(a)
    assert [a[n]._version for n in ("k_cache", "v_scales")] > versions
