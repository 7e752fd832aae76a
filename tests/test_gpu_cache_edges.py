"""The operators of a paged cache in 8 bits on the GPU where their range, their order or their larger forms end,
against the formulas in 64 bits (``cache_reference``) or what follows from them."""

import math
import os
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
from test_gpu_cache import _attend  # noqa: E402

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


# ---- attention: logits at the ends of FP32 ------------------------------------------------------------


def _one_row(heads, K, dtype, ps=64, D=64):
    """One query token at position 2 K over the positions 0 to K - 1 of a cache of its own."""
    pages = -(-K // ps)
    return dict(q=_randn((1, 1, heads, D), 1, dtype), k=_codes((pages, ps, 1, D), 2), v=_codes((pages, ps, 1, D), 3),
                indices=torch.arange(K, dtype=torch.int32, device=DEV).view(1, 1, K), query_positions=_ints([[2 * K]]),
                page_table=torch.arange(pages, dtype=torch.int32, device=DEV).view(1, pages),
                k_scales=_scales((pages, 1, 1), 4), v_scales=_scales((pages, 1, 1), 5), scale=D ** -0.5)


@pytest.mark.parametrize("heads,dtype", [(8, BF16), (16, FP16), (40, BF16)])
@pytest.mark.parametrize("slope", [1e6, 1e30])
@pytest.mark.parametrize("rows", [1, 200])
def test_attention_logits_far_below(heads, dtype, slope, rows):
    """The nearest entry's logit is -2e9 or -2e33, the next one's lower by 1e6 or 1e30: it has all the weight, whether
    CTAs share the row or not."""
    K = 2048
    c = _one_row(heads, K, dtype)
    c["slopes"] = torch.full((heads,), slope, device=DEV)
    for n in ("q", "indices", "query_positions", "page_table"):
        c[n] = c[n].expand(rows, *c[n].shape[1:]).contiguous()
    out, lse = tk.sparse_attention(**c, return_lse=True)
    want = R.np64(c["v"].float())[-1, -1, 0] * float(c["v_scales"][-1, 0, 0])
    assert np.abs(R.np64(out) - want).max() <= R.half_step(dtype) * np.abs(want).max()
    assert np.abs(R.np64(lse) / (-slope * (K + 1)) - 1).max() < 2.0 ** -20  # products and sums of FP32


@pytest.mark.parametrize("heads,dtype", [(8, BF16), (16, FP16), (64, BF16)])
@pytest.mark.parametrize("at", [5, 140, 290])
def test_attention_infinite_logits(heads, dtype, at):
    """One head's logit of one entry passes FP32's largest number, in the first tile or a later one: that head is NaN,
    and the others are what they are without."""
    K, D = 300, 64
    c = _one_row(heads, K, dtype, ps=1)
    c["q"][..., 0] = 0.0
    c["k"].view(torch.uint8)[at] = 0
    plain = tk.sparse_attention(**c, return_lse=True)
    c["q"][0, 0, 3, 0] = 16.0
    c["k"][at, 0, 0, 0] = 448.0
    c["k_scales"][at] = 2.0 ** 120  # 2^120 * 448 * 16 / 8, past 2^128 in units of log 2
    out, lse = tk.sparse_attention(**c, return_lse=True)
    assert torch.isnan(out[0, 0, 3]).all() and torch.isnan(lse[0, 0, 3])
    rest = [h for h in range(heads) if h != 3]
    assert torch.equal(out[0, 0, rest], plain[0][0, 0, rest]) and torch.equal(lse[0, 0, rest], plain[1][0, 0, rest])
    c["k"][at, 0, 0, 0] = -448.0  # a logit of -infinity has weight 0
    out, lse = tk.sparse_attention(**c, return_lse=True)
    hidden = c["indices"].clone()
    hidden[0, 0, at] = -1
    want = tk.sparse_attention(**{**c, "indices": hidden}, return_lse=True)
    assert torch.equal(out[0, 0, 3], want[0][0, 0, 3]) and torch.equal(lse[0, 0, 3], want[1][0, 0, 3])


# ---- attention: what small weights keep --------------------------------------------------------------


def _sink(heads, dtype, rows, n, fall, at, D=64, Dv=64):
    """One entry with a value of 0 at place `at`, n others with a value of 1 whose weights are 2^-fall of its."""
    q = torch.zeros((rows, 1, heads, D), dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    k = torch.zeros((n + 1, 1, 1, D), device=DEV)
    k[..., 0] = 256.0
    v = torch.ones((n + 1, 1, 1, Dv), device=DEV)
    v[at] = 0.0
    units = torch.full((n + 1, 1, 1), 2.0 ** -8, device=DEV)
    units[at] = (1.0 + fall * math.log(2.0)) * 2.0 ** -8
    c = dict(q=q, k=k.to(E4M3), v=v.to(E4M3), k_scales=units, v_scales=torch.ones_like(units), scale=1.0,
             indices=torch.arange(n + 1, dtype=torch.int32, device=DEV).expand(rows, 1, -1).contiguous())
    z = 256.0 * R.np64(units).ravel()
    p = np.exp(z - z.max())
    p /= p.sum()
    return c, 1.0 - p[at], p[at]


def _sink_bound(dtype, tail, top, n, fall, D=64):
    """What the header says of a weight: rounded to 9 bits or fp16, in steps of 2^-19 or 2^-23 of the largest one;
    logits and sums in FP32, the result rounded to its type."""
    rounded = 2.0 ** -11 if dtype == FP16 else 2.0 ** -9 + 2.0 ** -11
    step = 2.0 ** -23 if dtype == FP16 else 2.0 ** -19
    logits = (D + 16) * R.U * (2.0 + fall) + (n + 9) * R.U
    return tail * (rounded + 2.0 * logits + 1.01 * R.half_step(dtype)) + n * top * step / 2


@pytest.mark.parametrize("heads,dtype", [(8, BF16), (16, BF16), (64, BF16), (8, FP16), (32, FP16)])
@pytest.mark.parametrize("rows", [1, 320])
@pytest.mark.parametrize("at", [0, 1000, 2047])
def test_attention_one_entry_far_above_a_flat_rest(heads, dtype, rows, at):
    """An attention sink: one entry of no value has most of the weight, and the others' small weights are the result."""
    n = 2047
    for fall in (9.3, 12.2, 13.6, 14.5, 15.2, 16.4, 17.2, 17.6, 19.5, 21.6):
        c, tail, top = _sink(heads, dtype, rows, n, fall, at)
        out, lse = tk.sparse_attention(**c, return_lse=True)
        bound = _sink_bound(dtype, tail, top, n, fall)
        assert np.abs(R.np64(out) - tail).max() <= bound, f"{fall}: {np.abs(R.np64(out) - tail).max()} for {bound} of {tail}"


@pytest.mark.parametrize("heads,dtype", [(8, BF16), (64, BF16), (12, FP16), (32, FP16)])
@pytest.mark.parametrize("rows,n", [(1, 4095), (320, 4095), (320, 8190), (40, 16383), (200, 16383)])
def test_attention_long_lists(heads, dtype, rows, n):
    """The same beside lists past 2048 entries: what is lost beside the one entry is lost of 2048 entries at most."""
    for fall in (14.5, 17.6, 19.5, 20.7, 23.4):
        c, tail, top = _sink(heads, dtype, rows, n, fall, n // 3)
        out, lse = tk.sparse_attention(**c, return_lse=True)
        bound = _sink_bound(dtype, tail, top, n, fall) - (n - 2047) * top * (2.0 ** -23 if dtype == FP16 else 2.0 ** -19) / 2
        bound += 2 * tail * (n + 9) * R.U  # more sums in FP32, and the join
        assert np.abs(R.np64(out) - tail).max() <= bound, f"{fall}: {np.abs(R.np64(out) - tail).max()} for {bound} of {tail}"


# ---- append: tokens in any order ---------------------------------------------------------------------


def _prompts(counts, ps, seed, start=None):
    """(slots, positions, pages) of sequences of these many tokens each, from a place of their first page on."""
    g = np.random.default_rng(seed)
    pages = sum(-(-n // ps) + 1 for n in counts)
    order, slots, positions = list(g.permutation(pages + 2)), [], []
    for n in counts:
        at = int(g.integers(0, ps)) if start is None else start
        mine = [int(order.pop()) for _ in range((at + n - 1) // ps + 1)]
        slots.append([mine[w // ps] * ps + w % ps for w in range(at, at + n)])
        positions.append(list(range(at, at + n)))
    return slots, positions, pages + 2


def _steps(counts, lists):
    """Token by token over the sequences."""
    return [lists[b][i] for i in range(max(counts)) for b in range(len(counts)) if i < counts[b]]


def _append_case(slots, positions, pages, H, D, Dv, rotated, ps, blocks, dtype, seed=0):
    T = len(slots)
    grow = torch.exp2(torch.randint(-3, 4, (T, H, 1), generator=_gen(seed + 9), device=DEV).float())
    scaled = blocks > 0
    c = dict(k=(_randn((T, H, D), seed + 1) * grow).to(dtype), v=(_randn((T, H, Dv), seed + 2) * grow).to(dtype) if Dv else None,
             slots=_ints(slots), positions=_ints(positions), f=tk.rotary_frequencies(rotated, device=DEV) if rotated else None,
             v_cache=None, k_scales=None, v_scales=None)
    for i, (side, d) in enumerate((("k", D), ("v", Dv))):
        if d:
            shape = (pages, ps, H, d)
            c[side + "_cache"] = _codes(shape, seed + 3 + i) if scaled else _randn(shape, seed + 3 + i, dtype)
            c[side + "_scales"] = _scales((pages, blocks, H), seed + 5 + i) if scaled else None
    return c


def _append_check(c, layout="half", offset=0, scale=1.0):
    want = []
    for side in ("k", "v"):
        cache, scales = c[side + "_cache"], c[side + "_scales"]
        if cache is not None:
            block = cache.shape[1] // scales.shape[1] if scales is not None else 1
            want.append((side, *C.append(c[side], c["positions"], c["f"] if side == "k" else None, cache, scales, c["slots"],
                                         block, layout, offset, scale)))
    tk.cache_append(c["k"], c["v"], c["positions"], c["f"], c["k_cache"], c["v_cache"], c["slots"], k_scales=c["k_scales"],
                    v_scales=c["v_scales"], layout=layout, offset=offset, scale=scale)
    for side, cache, bound, scales in want:
        if scales is not None:
            assert np.array_equal(R.np64(c[side + "_scales"]), scales), f"{side} scales"
        R.assert_near(c[side + "_cache"].float(), cache, bound, side)


@pytest.mark.parametrize("order", ["steps", "idle", "shuffled"])
@pytest.mark.parametrize("counts,H,D,Dv,rotated,ps,blocks,dtype,layout", [
    ([2, 2], 2, 64, 64, 64, 16, 1, BF16, "half"),
    ([3] * 40, 3, 64, 48, 32, 64, 2, FP16, "half"),
    ([70, 1, 33], 5, 40, 18, 6, 12, 2, FP32, "interleaved"),
    ([130, 64, 65], 2, 128, 0, 128, 64, 1, BF16, "interleaved"),
    ([50, 20], 1, 64, 64, 0, 8, 8, BF16, "half"),  # a scale each
    ([400] * 13, 4, 64, 64, 64, 64, 1, BF16, "half"),  # large forms
    ([901, 700, 3, 1200], 9, 64, 64, 48, 48, 3, FP32, "interleaved"),
    ([2] * 1200, 9, 64, 64, 64, 1, 1, FP16, "half"),
])
def test_append_in_any_order(order, counts, H, D, Dv, rotated, ps, blocks, dtype, layout):
    """A block's tokens anywhere in the call: step by step over the sequences, with idle tokens between, or shuffled."""
    lists, where, pages = _prompts(counts, ps, len(counts), start=0 if ps == 1 else None)
    if order == "idle":
        slots = [s for mine in lists for one in mine for s in (one, -1)]
        positions = [s for mine in where for one in mine for s in (one, 0)]
    else:
        slots, positions = _steps(counts, lists), _steps(counts, where)
    if order == "shuffled":
        to = np.random.default_rng(1).permutation(len(slots))
        slots, positions = [slots[i] for i in to], [positions[i] for i in to]
    _append_check(_append_case(slots, positions, pages, H, D, Dv, rotated, ps, blocks, dtype), layout)


@pytest.mark.parametrize("T", [300, 6000])
def test_append_one_block_in_many_parts(T):
    """Two blocks' tokens by turns, of one from its last place to its first."""
    ps, H, D = T, 2, 64
    slots = [s for i in range(T // 2) for s in (T // 2 - 1 - i, T + i)]
    c = _append_case(slots, list(range(T)), 2, H, D, D, D, ps, 1, BF16)
    c["k"][T // 2] *= 64.0
    _append_check(c)
    first = {n: c[n].clone().view(torch.uint8) for n in ("k_cache", "v_cache", "k_scales", "v_scales")}
    for _ in range(3):  # the same tokens once more change nothing
        tk.cache_append(c["k"], c["v"], c["positions"], c["f"], c["k_cache"], c["v_cache"], c["slots"], k_scales=c["k_scales"],
                        v_scales=c["v_scales"])
        assert all(torch.equal(c[n].view(torch.uint8), b) for n, b in first.items())


def test_append_scales_that_overlap():
    """Scales share no memory with each other, the caches or the inputs."""
    H, D, ps, pages = 2, 64, 8, 4
    lists, where, _ = _prompts([6], ps, 1)
    base = _append_case(lists[0], where[0], pages, H, D, D, D, ps, 2, BF16)
    pool = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)

    def at(start, like):
        return pool[start:start + like.numel() * like.element_size()].view(like.dtype).view(like.shape)

    size = base["k_scales"].numel() * 4
    for name in ("k_scales", "v_scales"):
        other = "v_scales" if name == "k_scales" else "k_scales"
        for of in ("k", "v", "k_cache", "v_cache", "slots", "positions", "f", other):
            c = dict(base)
            c[of] = at(1024, base[of])
            end = 1024 + base[of].numel() * base[of].element_size()
            for start in (1024 - size + 8, end - 8):
                c[name] = at(start, base[name])
                with pytest.raises(ValueError, match="_scales must not overlap"):
                    tk.cache_append(c["k"], c["v"], c["positions"], c["f"], c["k_cache"], c["v_cache"], c["slots"],
                                    k_scales=c["k_scales"], v_scales=c["v_scales"])
    c = dict(base, k_scales=at(1024, base["k_scales"]), v_scales=at(1024 + size, base["v_scales"]))
    _append_check(c)  # one behind the other


def test_attention_scales_that_overlap_the_result():
    c = _one_row(8, 100, BF16)
    pool = torch.zeros(1 << 14, dtype=torch.uint8, device=DEV)
    out = pool[4096:4096 + 8 * 64 * 2].view(BF16).view(1, 1, 8, 64)
    want = tk.sparse_attention(**c)
    for name in ("k_scales", "v_scales"):
        for start in (4096 - 4, 4096 + 8 * 64 * 2 - 4):
            part = pool[start:start + 8].view(FP32).view(c[name].shape)
            with pytest.raises(ValueError, match="out must not overlap k_scales"):
                tk.sparse_attention(**{**c, name: part}, out=out)
        part = pool[4096 - 8:4096].view(FP32).view(c[name].shape)
        part.copy_(c[name])
        assert torch.equal(tk.sparse_attention(**{**c, name: part}, out=out), want)


# ---- the larger forms --------------------------------------------------------------------------------

MANY = [
    # rows, query heads, key heads, D, Dv, K, dtype, shared: one, two or three works a CTA, of one to five tiles
    (650, 8, 1, 64, 64, 130, BF16, False),
    (650, 16, 1, 128, 256, 300, BF16, False),
    (650, 16, 1, 256, 64, 129, FP16, True),
    (650, 12, 1, 128, 128, 260, FP16, False),
    (420, 32, 1, 192, 128, 400, BF16, False),
    (420, 24, 1, 128, 240, 300, FP16, False),
    (420, 32, 1, 256, 192, 520, FP16, True),
    (420, 64, 1, 256, 256, 300, BF16, False),  # one stage
    (420, 64, 1, 256, 192, 130, BF16, True),
    (420, 40, 1, 96, 80, 100, BF16, False),
    (210, 32, 4, 64, 128, 390, BF16, False),
    (170, 50, 1, 128, 80, 200, FP16, False),  # two tiles of heads
    (130, 35, 5, 96, 64, 300, FP16, False),
]


@pytest.mark.parametrize("rows,Hq,Hkv,D,Dv,K,dtype,shared", MANY)
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, True)])
def test_attention_several_rows_a_cta(rows, Hq, Hkv, D, Dv, K, dtype, shared, cap, bias):
    """More works than CTAs, the heads' logits of different sizes, so that in every tile some references move: a sample
    of the rows, first, second and third ones of their CTAs among them."""
    c = _attend(rows, 1, Hq, Hkv, D, Dv, K, 2 * K, 48, 3, dtype, seed=K + Hq, shared=shared)
    c["q"] = c["q"] * torch.exp2((torch.arange(Hq, device=DEV) * 5 % 7 - 3).float())[:, None].to(dtype)
    c["indices"][7] = -1  # a row that sees nothing, between others
    if bias:
        c["slopes"], c["softcap"] = _randn((Hq,), 6, FP32, 0.05), cap
    out, lse = tk.sparse_attention(**c, return_lse=True)
    assert torch.equal(out, tk.sparse_attention(**c))
    some = sorted({0, 7, 8, 151 % rows, 152 % rows, 153 % rows, 303 % rows, 304 % rows, 305 % rows, 455 % rows, 456 % rows,
                   608 % rows, 609 % rows, rows - 2, rows - 1})
    some = torch.tensor(some, device=DEV)
    pages = c["page_table"][some].flatten().long()
    clean = {n: torch.nan_to_num(c[n][pages].float(), nan=0.0) for n in ("k", "v", "k_scales", "v_scales")}
    table = torch.arange(pages.numel(), device=DEV).view(len(some), -1)
    want = C.attention(c["q"][some], clean["k"].to(E4M3), clean["v"].to(E4M3), clean["k_scales"], clean["v_scales"],
                       c["indices"][some], table, c["query_positions"][some], c["scale"], c.get("softcap", 0.0), c.get("slopes"))
    R.assert_near(lse[some], want[2], want[3], "lse")
    R.assert_near(out[some], want[0], want[1], "out")


LARGE = [
    # counts, H, D, Dv, rotated, offset, page size, blocks (0: of the inputs' type), dtype, layout
    ([1501, 800], 6, 128, 96, 128, 0, 64, 0, BF16, "half"),
    ([1501, 800], 9, 96, 128, 64, 32, 17, 0, FP16, "interleaved"),
    ([1401], 5, 128, 64, 96, 16, 64, 0, FP32, "half"),
    ([1000, 1], 3, 66, 18, 32, 2, 16, 0, BF16, "half"),  # nothing aligned
    ([1600, 1], 3, 33, 18, 32, 1, 16, 0, FP32, "interleaved"),
    ([2300, 33], 7, 128, 96, 64, 64, 64, 1, FP16, "half"),
    ([901, 700], 5, 112, 80, 48, 64, 48, 3, FP32, "interleaved"),
    ([901, 700], 5, 96, 64, 96, 0, 64, 4, FP32, "half"),
    ([1000, 3], 3, 65, 18, 32, 1, 16, 2, BF16, "interleaved"),  # nothing aligned
    ([1000, 3], 3, 66, 31, 30, 5, 16, 1, FP16, "half"),
    ([1500, 700], 7, 64, 128, 64, 0, 512, 1, BF16, "interleaved"),  # runs of several sweeps
    ([700, 500], 3, 512, 256, 512, 0, 64, 1, FP16, "half"),  # read twice
    ([300, 300], 2, 1024, 1000, 64, 960, 32, 1, FP32, "half"),
    ([400, 200], 1, 1023, 515, 1022, 1, 32, 2, BF16, "interleaved"),  # more items than threads
    ([3000, 2500], 9, 64, 0, 64, 0, 64, 64, BF16, "half"),  # keys alone, a scale each
]


@pytest.mark.parametrize("counts,H,D,Dv,rotated,offset,ps,blocks,dtype,layout", LARGE)
@pytest.mark.parametrize("idle", [False, True])
def test_append_large(counts, H, D, Dv, rotated, offset, ps, blocks, dtype, layout, idle):
    """Calls of as many tokens as prompts have, in all that the forms for them tell apart, idle tokens between or not."""
    lists, where, pages = _prompts(counts, ps, len(counts))
    slots, positions = sum(lists, []), sum(where, [])
    if idle:
        slots = [s for i, one in enumerate(slots) for s in ((one, -1) if i % 5 == 0 else (one,))]
        positions = [s for i, one in enumerate(positions) for s in ((one, 0) if i % 5 == 0 else (one,))]
    _append_check(_append_case(slots, positions, pages, H, D, Dv, rotated, ps, blocks, dtype), layout, offset, 0.75)


# ---- the example's step ------------------------------------------------------------------------------


@pytest.mark.parametrize("eight", [False, True])
def test_example_step_fills_its_caches(eight):
    """The step on caches of either kind against its plain form, and what it appended against the formulas."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import sparse_step as ex

    torch.manual_seed(4)
    cache, f, token = ex.make(5, 900, eight=eight)
    q, k, v, index_q, weights, index_k, lengths = token
    positions = lengths - 1
    slots, block = cache.slots(positions), 1 if not eight else None
    wants = [C.append(x, positions, turn, held, units, slots, block or held.shape[1] // units.shape[1])
             for x, turn, held, units in ((k, f, cache.k, cache.k_scales), (v, None, cache.v, cache.v_scales),
                                          (index_k[:, None], f, cache.index_k[:, :, None],
                                           None if not eight else cache.index_scales))]
    got = ex.step(cache, f, *token, 128)
    for (want, bound, _), held in zip(wants, (cache.k, cache.v, cache.index_k[:, :, None])):
        R.assert_near(held.float(), want, bound)
    plain = ex.step_plain(cache, f, *token, 128)
    # the queries' and the result's roundings and the weights', then a swapped entry
    assert (got - plain).float().norm() <= (3 * 2.0 ** -8 + 0.02) * plain.float().norm()


# ---- sines and cosines -------------------------------------------------------------------------------


@pytest.mark.parametrize("call", ["rotary", "cache_append"])
def test_small_sines_and_cosines(call):
    """Pairs (1, 0) turn to a cosine and a sine: in fp16, whose steps are small near zero, each is off by 2^-20 and its
    rounding at most."""
    T, pairs = 4000, 128
    f = torch.rand(pairs, dtype=torch.float64, generator=_gen(1), device=DEV) * 3.0
    positions = torch.randint(-(2 ** 20), 2 ** 20, (T,), generator=_gen(2), device=DEV)
    x = torch.zeros((T, 1, 2 * pairs), dtype=FP16, device=DEV)
    x[..., :pairs] = 1.0
    if call == "rotary":
        got = tk.rotary(x, positions, f)
    else:
        got = torch.zeros((1, T, 1, 2 * pairs), dtype=FP16, device=DEV)
        tk.cache_append(x, None, positions, f, got, None, torch.arange(T, dtype=torch.int32, device=DEV))
    angle = R.npi(positions).astype(np.longdouble)[:, None] * R.np64(f).astype(np.longdouble)
    want = np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float64)
    off = np.abs(R.np64(got).reshape(T, -1) - want)
    assert (off <= 2.0 ** -20 + (np.abs(want) + 2.0 ** -20) * 2.0 ** -11 + 2.0 ** -25).all()
    near = np.abs(want) < 2.0 ** -9
    assert near.sum() > 1000
    print(f"off by 2^{np.log2(off[near].max()):.2f} near zero")
