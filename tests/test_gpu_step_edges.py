"""The operators around the selection at the edges of what they accept, against their formulas in 64 bits."""

import ctypes
import math
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_attention_indexer_fp32_gb300 as tk  # noqa: E402
from sparse_attention_indexer_fp32_gb300 import _step  # noqa: E402

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


# ---- attention: the cap ------------------------------------------------------------------------------


def _capped(q, k, v, scale, cap):
    """(out, its bound, lse, its bound) of one row over all entries, [H, D] and [n, D]. A logit is off by
    its product's sum and its own rounding, and by 8 U of its capped value, whatever the cap; the rest as in
    step_reference.attention."""
    hs, U = R.half_step(v.dtype), R.U
    tiny = torch.finfo(v.dtype).tiny * torch.finfo(v.dtype).eps
    q, k, v = R.np64(q), R.np64(k), R.np64(v)
    cap = float(np.float32(cap))
    x = q @ k.T * scale
    z = cap * np.tanh(x / cap)
    slope = 1.0 - np.tanh(x / cap) ** 2
    dz = slope * ((q.shape[1] + 4) * U * abs(scale) * (np.abs(q) @ np.abs(k).T) + 4 * U * np.abs(x)) + 8 * U * np.abs(z)
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - top)
    total = e.sum(axis=1, keepdims=True)
    p = e / total
    dz = dz + 4 * U * np.abs(z - top) + 8 * U
    mean_dz = (p * dz).sum(axis=1) + (len(k) + 8) * U
    out = p @ v
    err = ((p * (hs + dz + mean_dz[:, None])) @ np.abs(v)) * 1.01 + tiny * np.abs(v).sum(axis=0) / total \
        + hs * np.abs(out) * 1.01 + tiny
    lse = (np.log(total) + top)[:, 0]
    return out, err, lse, mean_dz + 4 * U * (np.abs(top[:, 0]) + np.abs(lse))


@pytest.mark.parametrize("cap", [1e-40, 1e-30, 1e-3, 0.7, 5.0, 50.0, 1e4, 1e6, 1e8, 1e30, 3.4e38])
@pytest.mark.parametrize("heads", [6, 40, 80])
def test_attention_caps_of_any_size(cap, heads):
    """The cap's error goes with the logit, not with the cap: far above the logits it changes nothing."""
    n, D, ps = 150, 64, 16
    pages = -(-n // ps)
    q = _randn((1, 1, heads, D), 1, BF16, 2.0)
    k, v = (_randn((pages, ps, 1, D), s, BF16) for s in (2, 3))
    k[0, 3] = 0.0  # a logit of exactly 0
    idx = torch.arange(n, dtype=torch.int32, device=DEV).view(1, 1, n)
    out, lse = tk.sparse_attention(q, k, v, idx, softcap=cap, scale=0.25, return_lse=True)
    want = _capped(q[0, 0], k.view(-1, D)[:n], v.view(-1, D)[:n], 0.25, cap)
    R.assert_near(out[0, 0], want[0], want[1], "out")
    R.assert_near(lse[0, 0], want[2], want[3], "lse")


def test_attention_cap_under_the_smallest_number():
    """A positive cap that FP32 cannot hold is refused, not taken for no cap."""
    q = _randn((1, 1, 2, 64), 1, BF16)
    k = _randn((4, 16, 1, 64), 2, BF16)
    with pytest.raises(ValueError, match="softcap"):
        tk.sparse_attention(q, k, k, _ints([[[0, 1]]]), softcap=1e-60)


# ---- attention: infinities ----------------------------------------------------------------------------


@pytest.mark.parametrize("heads", [4, 40, 80])
def test_attention_infinities_that_are_seen(heads):
    """Infinite logits by the formula: the cap's ends, weight 0, NaN; an infinite value stays in its column."""
    n, D, ps = 100, 64, 16
    q = _randn((1, 1, heads, D), 1, BF16)
    q[..., 3] = q[..., 3].abs() + 0.1
    k, v = (_randn((7, ps, 1, D), s, BF16) for s in (2, 3))
    idx = torch.arange(n, dtype=torch.int32, device=DEV).view(1, 1, n)

    def call(k, v, idx=idx, **kw):
        return tk.sparse_attention(q, k, v, idx, return_lse=True, **kw)

    low, high = k.clone(), k.clone()
    low.view(-1, D)[70, 3], high.view(-1, D)[70, 3] = -math.inf, math.inf
    rest = torch.cat([idx[..., :70], idx[..., 71:]], dim=-1).contiguous()
    want = R.attention(q, k, v, rest, None, None, D ** -0.5, 0.0, None, None)
    got = call(low, v)
    R.assert_near(got[0], want[0], want[1])
    R.assert_near(got[1], want[2], want[3])
    assert all(torch.isnan(t).all() for t in call(high, v))
    out, lse = call(low, v, idx[..., 70:71].contiguous())
    assert (out == 0).all() and torch.isneginf(lse).all()
    only = torch.zeros_like(k)  # logits past any cap, then so far past it that they are it
    only.view(-1, D)[70, 3], only.view(-1, D)[71, 3] = -math.inf, math.inf
    far = only.nan_to_num(posinf=1e30, neginf=-1e30)
    for g, w in zip(call(only, v, softcap=2.0), call(far, v, softcap=2.0)):
        assert torch.equal(g, w) and torch.isfinite(g).all()
    value = v.clone()
    value.view(-1, D)[50, 9] = math.inf
    out, lse = call(k, value)
    plain, want = call(k, v)
    assert not torch.isfinite(out[..., 9]).any() and torch.equal(lse, want)
    keep = [d for d in range(D) if d != 9]
    assert torch.equal(out[..., keep], plain[..., keep])


# ---- indexer scores: infinite keys -------------------------------------------------------------------


@pytest.mark.parametrize("H", [1, 3, 8, 10, 16, 24, 32, 33, 48, 64, 65, 100, 128])
@pytest.mark.parametrize("T,ps,dtype", [(1, 64, BF16), (5, 7, FP16)])
def test_scores_of_infinite_keys(H, T, ps, dtype):
    """The formula's own infinities and zeros, whatever the number of heads."""
    width, D = 150, 64
    pages = -(-width // ps)
    keys = _randn((pages, ps, D), 1, dtype)
    q = _randn((1, T, H, D), 2, dtype)
    q[..., 3] = q[..., 3].abs() + 0.1
    w = _randn((1, T, H), 3).abs() + 0.1
    flat = keys.view(-1, D)
    flat[5, 3] = math.inf     # every product +inf
    flat[70, 3] = -math.inf   # every product -inf: nothing is added
    flat[140, 3], flat[140, 4] = math.inf, math.nan
    n = torch.full((1, T), width, dtype=torch.int32, device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    got = tk.indexer_scores(q, w, keys, n, table, width=width)
    assert (got[..., 5] == math.inf).all() and (got[..., 70] == 0.0).all() and torch.isnan(got[..., 140]).all()
    assert (tk.indexer_scores(q, -w, keys, n, table, width=width)[..., 5] == -math.inf).all()
    want, bound = R.scores(q, w, keys, n, table, None, width)
    keep = [s for s in range(width) if s not in (5, 70, 140)]
    R.assert_near(got[..., keep], want[..., keep], bound[..., keep])


# ---- rotary: rates ------------------------------------------------------------------------------------

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def test_rotary_fast_rates_at_far_positions():
    """Rates up to the limit of 2^40 radians a position, at both ends of 32 bits: the angle is that of the
    exact product. 2^-32 turns of the fraction, 2 ulp of the functions and three roundings: 16 U."""
    rates = [1.0, 0.1, 12345.678, 3.0e5, -(2.0 ** 30) * 1.1, 2.0 ** 35 + 0.37, 1.3 * 2.0 ** 39, 2.0 ** -30]
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 77, -1]
    x = _randn((len(pos), 3, 2 * len(rates)), 1)
    f = torch.tensor(rates, dtype=torch.float64, device=DEV)
    got = R.np64(tk.rotary(x, _ints(pos), f))
    angle = np.array([[float((Fraction(r) * p / TWO_PI) % 1) for r in rates] for p in pos]) * 2 * math.pi
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    u, v = np.split(R.np64(x), 2, axis=-1)
    want = np.concatenate([u * c - v * s, v * c + u * s], axis=-1)
    R.assert_near(got, want, np.tile(16 * R.U * np.hypot(u, v), 2))


# ---- errors left behind -------------------------------------------------------------------------------


def test_an_earlier_failure_is_not_reported_again():
    """A call whose launch is refused (the legacy stream while another stream that waits for it is being captured)
    reports it, and the next calls, whose launches go through, do not."""
    cuda = ctypes.CDLL("libcuda.so.1")
    f, pos = tk.rotary_frequencies(64, device=DEV), _ints([1, 2])
    x = _randn((2, 4, 64), 1, BF16)
    k = _randn((4, 16, 1, 64), 2, BF16)
    idx, table, n = _ints([[[0, 5, 9]], [[1, 2, 3]]]), _ints([[0, 1], [2, 3]]), _ints([[20], [32]])
    w = _randn((2, 1, 4), 3)
    bufs = torch.empty_like(x), torch.empty((2, 1, 32), device=DEV), torch.empty((2, 1, 4, 64), dtype=BF16, device=DEV)

    def rotary():
        return tk.rotary(x, pos, f, out=bufs[0])

    def scores():
        return tk.indexer_scores(x[:, None], w, k[:, :, 0], n, table, out=bufs[1])

    def attention():
        return tk.sparse_attention(x[:, None], k, k, idx, table, out=bufs[2])

    for call in (rotary, scores, attention):
        call()
    torch.cuda.synchronize()
    for failing in (rotary, scores, attention):
        stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
        assert cuda.cuStreamCreate(ctypes.byref(stream), 0) == 0
        try:
            assert cuda.cuStreamBeginCapture_v2(stream, 0) == 0
            try:
                with pytest.raises(tk.TopkError):
                    failing()
            finally:
                cuda.cuStreamEndCapture(stream, ctypes.byref(graph))
        finally:
            assert cuda.cuStreamDestroy_v2(stream) == 0
        for call in (rotary, scores, attention):
            call()
        torch.cuda.synchronize()


# ---- dimensions of one ---------------------------------------------------------------------------------


def test_strides_of_single_elements_do_not_matter():
    """A stride that no element is reached by may be anything."""
    D, ps, n = 64, 32, 20
    q = _randn((1, 1, 6, D), 1, BF16)
    k = _randn((1, ps, 1, D), 2, BF16)
    odd = k.as_strided(k.shape, (3, D, 5, 1))
    idx, table, length = torch.arange(n, dtype=torch.int32, device=DEV).view(1, 1, n), _ints([[0]]), _ints([[n]])
    assert torch.equal(tk.sparse_attention(q, odd, odd, idx, table), tk.sparse_attention(q, k, k, idx, table))
    w = _randn((1, 1, 6), 3)
    want = tk.indexer_scores(q, w, k[:, :, 0], length, table)
    assert torch.equal(tk.indexer_scores(q, w, odd[:, :, 0], length, table)[..., :n], want[..., :n])
    single = k[:, :1].as_strided((1, 1, 1, D), (3, 7, 5, 1))  # pages of one entry
    assert torch.equal(tk.sparse_attention(q, single, single, idx[..., :1].contiguous(), table),
                       tk.sparse_attention(q, k[:, :1], k[:, :1], idx[..., :1].contiguous(), table))
    f, pos = tk.rotary_frequencies(D, device=DEV), _ints([7])
    x = _randn((1, 3, D), 4, BF16)
    want = tk.rotary(x, pos, f)
    strange = x.as_strided(x.shape, (1, D, 1))
    assert torch.equal(tk.rotary(strange, pos, f), want)
    assert tk.rotary(strange, pos, f, out=x) is x and torch.equal(x, want)  # in place through another view of it


# ---- autograd -----------------------------------------------------------------------------------------


def test_nothing_that_needs_a_gradient_is_taken():
    """Where gradients are recorded the calls refuse what would need one; without, they run."""
    f, pos = tk.rotary_frequencies(64, device=DEV), _ints([1, 2])
    x, w = _randn((2, 4, 64), 1, BF16), _randn((2, 1, 4), 3)
    k = _randn((4, 16, 1, 64), 2, BF16)
    idx, table, n = _ints([[[0, 5, 9]], [[1, 2, 3]]]), _ints([[0, 1], [2, 3]]), _ints([[20], [32]])
    slopes, qpos = torch.zeros(4, device=DEV), _ints([[9], [9]])

    def leaf(t):
        return t.clone().requires_grad_()

    calls = [lambda: tk.rotary(leaf(x), pos, f), lambda: tk.rotary(x, pos, f, out=leaf(x)),
             lambda: tk.indexer_scores(leaf(x[:, None]), w, k[:, :, 0], n, table),
             lambda: tk.indexer_scores(x[:, None], leaf(w), k[:, :, 0], n, table),
             lambda: tk.indexer_scores(x[:, None], w, leaf(k[:, :, 0]), n, table),
             lambda: tk.sparse_attention(leaf(x[:, None]), k, k, idx, table),
             lambda: tk.sparse_attention(x[:, None], leaf(k), k, idx, table),
             lambda: tk.sparse_attention(x[:, None], k, leaf(k), idx, table),
             lambda: tk.sparse_attention(x[:, None], k, k, idx, table, slopes=leaf(slopes), query_positions=qpos)]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad():
            call()


def test_a_tensor_written_in_place_is_known_to_have_changed():
    """A backward pass that needs what `out` held before is refused by autograd, not run on the new values."""
    f, pos = tk.rotary_frequencies(64, device=DEV), _ints([1, 2])
    x, k = _randn((2, 4, 64), 1, BF16), _randn((4, 16, 1, 64), 2, BF16)
    w, scores = _randn((2, 1, 4), 3), torch.zeros((2, 1, 32), device=DEV)
    idx, table, n = _ints([[[0, 5, 9]], [[1, 2, 3]]]), _ints([[0, 1], [2, 3]]), _ints([[20], [32]])
    out = torch.zeros((2, 1, 4, 64), dtype=BF16, device=DEV)
    for target, call in ((x, lambda: tk.rotary(x, pos, f, out=x)),
                         (k, lambda: tk.rotary(x[:, :1], pos, f, out=k, slots=_ints([3, 4]))),
                         (scores, lambda: tk.indexer_scores(x[:, None], w, k[:, :, 0], n, table, out=scores)),
                         (out, lambda: tk.sparse_attention(x[:, None], k, k, idx, table, out=out))):
        weight = torch.ones_like(target, requires_grad=True)
        loss = (target * weight).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():  # whose tensors have no version
        y = x.clone()
        assert torch.equal(tk.rotary(y, pos, f, out=y), tk.rotary(x, pos, f))


# ---- the longest ---------------------------------------------------------------------------------------


def test_attention_over_the_longest_list():
    """2^31 - 1 indices (8.6 GB), all but a few of them of nothing."""
    K, D = 2 ** 31 - 1, 64
    idx = torch.full((1, 1, K), -1, dtype=torch.int32, device=DEV)
    at = [0, 63, 64, 2 ** 30, K - 65, K - 64, K - 1]
    idx[0, 0, at] = torch.arange(len(at), dtype=torch.int32, device=DEV)
    q, k = _randn((1, 1, 2, D), 1, BF16), _randn((1, 16, 1, D), 2, BF16)
    short = torch.arange(len(at), dtype=torch.int32, device=DEV).view(1, 1, -1)
    got, lse = tk.sparse_attention(q, k, k, idx, return_lse=True)
    want = R.attention(q, k, k, short, None, None, D ** -0.5, 0.0, None, None)
    R.assert_near(got, want[0], want[1])
    R.assert_near(lse, want[2], want[3])


def test_scores_of_the_most_tokens():
    """2^31 - 1 query tokens of one sequence, one score each (26 GB)."""
    T, D = 2 ** 31 - 1, 16
    q, keys = _randn((1, 1, 1, D), 1, BF16), _randn((1, 1, D), 2, BF16)
    if float(q.float().flatten() @ keys.float().flatten()) < 0:
        q = -q
    w = torch.ones((1, T, 1), device=DEV)
    n = torch.ones((1, T), dtype=torch.int32, device=DEV)
    out = torch.zeros((1, T, 1), device=DEV)
    tk.indexer_scores(q.expand(1, T, 1, D), w, keys, n, _ints([[0]]), out=out)
    few = tk.indexer_scores(q, w[:, :1], keys, n[:, :1], _ints([[0]]))
    assert (out == few).all()


def test_scores_of_too_many_units_are_refused():
    some, most = torch.zeros(64, device=DEV), 2 ** 31 - 1
    lib = tk.load_library()
    fn, kind = lib.sparse_indexer_scores, _step._ScoresArgs
    fn.argtypes, fn.restype = [ctypes.POINTER(kind), ctypes.c_void_p], ctypes.c_int
    for sizes in (dict(B=most, T=most, width=64, table_width=64), dict(B=most, T=most, width=most, table_width=most),
                  dict(B=most, T=1, width=most, table_width=most)):
        a = kind(q=some.data_ptr(), q_seq_stride=0, q_token_stride=0, q_head_stride=0, weights=some.data_ptr(),
                 keys=some.data_ptr(), key_page_stride=0, key_token_stride=0, lengths=some.data_ptr(),
                 page_table=some.data_ptr(), out=some.data_ptr(), num_pages=1, page_size=1, H=1, D=16, **sizes)
        assert fn(ctypes.byref(a), None) == tk.Status.EINVAL, sizes


# ---- waits that run out --------------------------------------------------------------------------------


@pytest.fixture(scope="module")
def hurried(tmp_path_factory):
    """The library once more, with waits that give up at once or after 3 us: {limit in ns: {call: its function}}."""
    from sparse_attention_indexer_fp32_gb300 import build as cuda_build

    units = ["step_abi.cu", "rotary.cu", "sparse_attention.cu", "indexer_scores_bf16.cu", "indexer_scores_fp16.cu",
             "indexer_scores_e4m3.cu"]
    out = tmp_path_factory.mktemp("hurried")
    jobs = []
    for ns in (0, 3000):
        for u in units:
            jobs.append(subprocess.Popen([cuda_build.nvcc(), *cuda_build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                                          "-I", cuda_build.INCLUDE, f"-DSPARSE_WAIT_LIMIT_NS={ns}", "-c",
                                          os.path.join(cuda_build.CSRC, u), "-o", str(out / f"{ns}_{u}.o")]))
    assert [job.wait() for job in jobs] == [0] * len(jobs)
    calls = {}
    for ns in (0, 3000):
        path = str(out / f"libhurried_{ns}.so")
        subprocess.check_call([cuda_build.nvcc(), *cuda_build.ARCH, "-shared", "-o", path,
                               *(str(out / f"{ns}_{u}.o") for u in units)])
        lib = ctypes.CDLL(path)
        prototype = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, ctypes.c_void_p)
        calls[ns] = {call: prototype(ctypes.cast(getattr(lib, call.name), ctypes.c_void_p).value)
                     for call in (_step._scores, _step._attention)}
    return calls


def _right_or_nan(hurried, monkeypatch, call):
    """With waits that run out each number is what it is without, or NaN, and the calls after are right again."""
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


@pytest.mark.parametrize("B,T,H,ps,dtype", [(2, 1, 64, 64, BF16), (3, 5, 24, 7, FP16), (200, 1, 32, 64, BF16),
                                            (1, 300, 16, 16, E4M3), (1, 64, 128, 64, BF16)])
def test_scores_whose_waits_run_out(hurried, monkeypatch, B, T, H, ps, dtype):
    width, D = 2300, 64
    pages = -(-width // ps)
    q, w = _randn((B, T, H, D), 1).to(dtype), _randn((B, T, H), 2)
    keys = _randn((B * pages, ps, D), 3).to(dtype)
    table = torch.arange(B * pages, dtype=torch.int32, device=DEV).view(B, pages)
    n = torch.randint(0, width + 1, (B, T), generator=_gen(4), device=DEV).to(torch.int32)
    _right_or_nan(hurried, monkeypatch,
                  lambda: (tk.indexer_scores(q, w, keys, n, table, out=torch.full((B, T, width), 7.0, device=DEV)),))


@pytest.mark.parametrize("rows,Hq,Hkv,K,shared", [(1, 8, 1, 2048, False), (3, 16, 4, 700, True), (100, 8, 4, 300, False),
                                                  (2, 40, 1, 900, False), (340, 40, 1, 130, False), (340, 70, 1, 64, True),
                                                  (20, 150, 1, 200, False)])
def test_attention_whose_waits_run_out(hurried, monkeypatch, rows, Hq, Hkv, K, shared):
    D, ps = 64, 16
    q, k = _randn((rows, 1, Hq, D), 1, BF16), _randn((200, ps, Hkv, D), 2, BF16)
    v = k if shared else _randn(k.shape, 3, BF16)
    idx = torch.randint(-1, 200 * ps, (rows, 1, K), generator=_gen(4), device=DEV).to(torch.int32)
    _right_or_nan(hurried, monkeypatch, lambda: tk.sparse_attention(q, k, v, idx, softcap=30.0, return_lse=True))


# ---- two streams ---------------------------------------------------------------------------------------


def test_scores_and_attention_side_by_side():
    """Kernels of both calls, with all or half of an SM's TMEM, with clusters and without, on two streams at once."""
    q, k = _randn((40, 1, 32, 128), 1, BF16), _randn((300, 16, 4, 128), 2, BF16)
    idx = torch.randint(-1, 4800, (40, 1, 600), generator=_gen(3), device=DEV).to(torch.int32)
    wide, entry = _randn((3, 1, 40, 256), 4, BF16), _randn((300, 16, 1, 256), 5, BF16)
    some = torch.randint(-1, 4800, (3, 1, 900), generator=_gen(6), device=DEV).to(torch.int32)
    iq, w = _randn((16, 1, 32, 64), 7, BF16), _randn((16, 1, 32), 8)
    keys, table = k.view(300, 16, 8, 64)[:, :, 0], torch.arange(300, dtype=torch.int32, device=DEV).expand(16, -1)
    n = torch.full((16, 1), 4800, dtype=torch.int32, device=DEV)
    calls = [lambda: tk.sparse_attention(q, k, k, idx), lambda: tk.indexer_scores(iq, w, keys, n, table),
             lambda: tk.sparse_attention(wide, entry, entry, some), lambda: tk.sparse_attention(q[:2], k, k, idx[:2]),
             lambda: tk.indexer_scores(iq[:3], w[:3], keys, n[:3], table[:3])]
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
