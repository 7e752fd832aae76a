"""ctypes binding of the operators around the selection (``include/sparse_step.h``).

As in ``_binding``: tensors are checked here, the rest by the library; every
step runs in its CUDA kernels, on the stream given or the current one, and
there is no CPU fallback.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _binding

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class _RotaryArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_token_stride", _i64), ("x_head_stride", _i64), ("out", _vp),
                ("out_page_stride", _i64), ("out_token_stride", _i64), ("out_head_stride", _i64),
                ("positions", _vp), ("frequencies", _vp), ("slots", _vp), ("num_pages", _i64),
                ("page_size", _i32), ("T", _i32), ("H", _i32), ("D", _i32), ("rotated", _i32),
                ("offset", _i32), ("layout", _i32), ("type", _i32), ("positions_64", _i32),
                ("inverse", _i32), ("scale", _f32)]


class _ScoresArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_seq_stride", _i64), ("q_token_stride", _i64), ("q_head_stride", _i64),
                ("weights", _vp), ("keys", _vp), ("key_page_stride", _i64), ("key_token_stride", _i64),
                ("key_scales", _vp), ("lengths", _vp), ("page_table", _vp), ("table_stride", _i64),
                ("table_width", _i64), ("out", _vp), ("out_seq_stride", _i64), ("out_token_stride", _i64),
                ("num_pages", _i64), ("width", _i64), ("page_size", _i32), ("B", _i32), ("T", _i32),
                ("H", _i32), ("D", _i32), ("type", _i32)]


class _AttentionArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_seq_stride", _i64), ("q_token_stride", _i64), ("q_head_stride", _i64),
                ("k", _vp), ("k_page_stride", _i64), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v", _vp), ("v_page_stride", _i64), ("v_token_stride", _i64), ("v_head_stride", _i64),
                ("indices", _vp), ("page_table", _vp), ("table_stride", _i64), ("table_width", _i64),
                ("query_positions", _vp), ("first", _vp), ("slopes", _vp), ("out", _vp), ("lse", _vp),
                ("num_pages", _i64), ("page_size", _i32), ("B", _i32), ("T", _i32), ("Hq", _i32),
                ("Hkv", _i32), ("D", _i32), ("Dv", _i32), ("K", _i32), ("type", _i32), ("scale", _f32),
                ("softcap", _f32)]


_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
_LAYOUTS = {"half": 0, "interleaved": 1}
_functions = {}


def _function(name: str, args):
    """The library's entry point ``name``, its signature set on first use."""
    fn = _functions.get(name)
    if fn is None:
        fn = getattr(_binding.load_library(), name)
        fn.argtypes = [ctypes.POINTER(args), _vp]
        fn.restype = ctypes.c_int
        _functions[name] = fn
    return fn


def _call(name: str, args, index: int, stream) -> None:
    fn = _function(name, type(args))
    sh = _binding._stream_handle(index, stream)
    status = _binding._on_device(index, lambda: fn(ctypes.byref(args), sh))
    if status != _binding.Status.OK:
        message = _binding.load_library().topk_status_string(status).decode()
        raise _binding.TopkError(status, f"{name} failed: {message}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _tensor(t, name: str, dims: int, dtypes, device=None) -> None:
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-D tensor")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor on the device of the other arguments")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, not {t.dtype}")


def _unit_inner(t: torch.Tensor, name: str) -> None:
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")


def _exact(t, name: str, shape, dtypes, device) -> None:
    """A contiguous tensor of exactly this shape."""
    _tensor(t, name, len(shape), dtypes, device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {list(shape)}")


def _span(t: torch.Tensor):
    """The bytes [start, end) that the elements of ``t`` lie within."""
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) if t.numel() else -1
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    (a0, a1), (b0, b1) = _span(a), _span(b)
    return a0 < b1 and b0 < a1


def _no_self_overlap(t: torch.Tensor, name: str) -> None:
    """An output may not be a broadcast: two of its elements at one address."""
    if any(s == 0 and n > 1 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{name} must not be a broadcast tensor")


def rotary_frequencies(rotated: int, base: float = 10000.0, *, scaling: Optional[str] = None,
                       factor: float = 1.0, original_length: int = 4096, fast: float = 32.0,
                       slow: float = 1.0, device="cuda") -> torch.Tensor:
    """Radians per position of each of ``rotated // 2`` pairs, ``base ** (-2 i / rotated)``, float64
    on ``device``, for :func:`rotary`.

    ``scaling`` stretches a context of ``original_length`` positions by ``factor``: ``"linear"``
    divides every frequency by it; ``"base"`` raises the base to ``base * factor ** (rotated /
    (rotated - 2))``, which keeps the fastest pair and divides the slowest by the factor; ``"ramp"``
    keeps pairs that turn more than ``fast`` times within ``original_length``, divides those that turn
    less than ``slow`` times, and blends linearly over the pairs between (the by-parts interpolation of
    the YaRN paper, Peng et al. 2023, section 3.2; its section 3.3 goes with ``scale = 0.1 *
    math.log(factor) + 1`` in :func:`rotary`)."""
    if rotated < 2 or rotated % 2:
        raise ValueError("rotated must be an even number, at least 2")
    if not (base > 0.0 and math.isfinite(base)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("base must be positive and factor at least 1, both finite")
    i = torch.arange(rotated // 2, dtype=torch.float64)
    if scaling == "base":
        if rotated < 4:
            raise ValueError("the base is scaled for at least two pairs")
        base = base * factor ** (rotated / (rotated - 2))
    f = base ** (-2.0 * i / rotated)
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        if original_length < 1 or not fast > slow > 0.0:
            raise ValueError("the ramp needs original_length >= 1 and fast > slow > 0")
        if base == 1.0:
            raise ValueError("the ramp needs a base other than 1")

        def pair(turns: float) -> float:  # the (fractional) pair that turns so often
            return rotated * math.log(original_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        low = min(max(math.floor(pair(fast)), 0), rotated // 2 - 1)
        high = min(max(math.ceil(pair(slow)), 0), rotated // 2 - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        f = f * (1.0 - ramp) + f / factor * ramp
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'ramp'")
    return f.to(device)


def rotary(x: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor, *, layout: str = "half",
           offset: int = 0, scale: float = 1.0, inverse: bool = False, out: Optional[torch.Tensor] = None,
           slots: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotary positions: the ``2 * len(frequencies)`` elements of every head of ``x`` from ``offset``
    on, turned pair by pair by ``positions[t] * frequencies[i]`` radians and multiplied by ``scale``;
    the rest of the head is copied.

    ``x`` bfloat16, float16 or float32 ``[T, H, D]`` (any strides, unit in ``D``, e.g. a slice of a
    joint query-key-value tensor), ``positions`` int32 or int64 ``[T]``, ``frequencies`` float64 on
    the GPU (:func:`rotary_frequencies`). ``layout`` ``"half"`` pairs element ``i`` with ``i +
    rotated / 2``, ``"interleaved"`` ``2 i`` with ``2 i + 1``. ``inverse`` turns back: the gradient
    of the call with the same arguments. ``out`` may be ``x`` (in place). With ``slots`` (int32
    ``[T]``), ``out`` is a paged cache ``[pages, page_size, H, D]`` and token ``t`` is written at slot
    ``slots[t]`` (negative or past the cache: not written). Returns ``out``."""
    _tensor(x, "x", 3, (torch.bfloat16, torch.float16, torch.float32))
    _unit_inner(x, "x")
    T, H, D = x.shape
    _exact(positions, "positions", (T,), (torch.int32, torch.int64), x.device)
    _tensor(frequencies, "frequencies", 1, (torch.float64,), x.device)
    if not frequencies.is_contiguous():
        raise ValueError("frequencies must be contiguous")
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    a = _RotaryArgs()
    if slots is None:
        if out is None:
            out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
        _tensor(out, "out", 3, (x.dtype,), x.device)
        if out.shape != x.shape:
            raise ValueError("out must have the shape of x")
    else:
        if out is None:
            raise ValueError("slots need the cache as out")
        _tensor(out, "out", 4, (x.dtype,), x.device)
        if tuple(out.shape[2:]) != (H, D):
            raise ValueError("out must be a cache [pages, page_size, H, D]")
        _exact(slots, "slots", (T,), (torch.int32,), x.device)
        a.slots, a.num_pages, a.page_size = slots.data_ptr(), out.shape[0], out.shape[1]
        a.out_page_stride = out.stride(0)
    _unit_inner(out, "out")
    _no_self_overlap(out, "out")
    same = slots is None and out.data_ptr() == x.data_ptr() and out.stride() == x.stride()
    if not same and _overlap(x, out):
        raise ValueError("out must be x itself or not overlap it")
    a.x, a.x_token_stride, a.x_head_stride = x.data_ptr(), x.stride(0), x.stride(1)
    a.out, a.out_token_stride, a.out_head_stride = out.data_ptr(), out.stride(-3), out.stride(-2)
    a.positions, a.positions_64 = positions.data_ptr(), int(positions.dtype == torch.int64)
    a.frequencies, a.rotated, a.offset = frequencies.data_ptr(), 2 * frequencies.numel(), int(offset)
    a.T, a.H, a.D, a.layout, a.type = T, H, D, _LAYOUTS[layout], _TYPES[x.dtype]
    a.inverse, a.scale = int(bool(inverse)), float(scale)
    _call("sparse_rotary", a, x.get_device(), stream)
    return out


def indexer_scores(q: torch.Tensor, weights: torch.Tensor, keys: torch.Tensor, lengths: torch.Tensor,
                   page_table: torch.Tensor, *, key_scales: Optional[torch.Tensor] = None,
                   width: Optional[int] = None, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The indexer's scores over a paged key cache: ``out[b, t, s] = key_scales[e] * sum_h weights[b, t,
    h] * max(0, q[b, t, h] . keys[e])`` for the entry ``e`` of every position ``s < lengths[b, t]`` of
    sequence ``b``; positions from the length on are not written.

    ``q`` ``[B, T, H, D]`` (T query tokens a sequence: 1 to decode, a prompt's tokens with their own
    causal lengths to prefill) and ``keys`` ``[pages, page_size, D]`` both bfloat16, float16 or
    float8_e4m3fn (the queries' scales then belong into ``weights``, the keys' into ``key_scales``,
    float32 ``[pages, page_size]``); ``weights`` float32 ``[B, T, H]``; ``lengths`` int32 ``[B, T]``;
    ``page_table`` int32 ``[B, n]`` (rows may be a broadcast). ``out`` float32 ``[B, T, width]``
    (default width: ``n * page_size``); ``out.view(B * T, width)`` is what :func:`topk_ragged`
    takes."""
    types = (torch.bfloat16, torch.float16, torch.float8_e4m3fn)
    _tensor(q, "q", 4, types)
    _unit_inner(q, "q")
    B, T, H, D = q.shape
    _exact(weights, "weights", (B, T, H), (torch.float32,), q.device)
    _tensor(keys, "keys", 3, (q.dtype,), q.device)
    _unit_inner(keys, "keys")
    if keys.shape[2] != D:
        raise ValueError("keys must have the head size of q")
    pages, page_size = keys.shape[:2]
    _exact(lengths, "lengths", (B, T), (torch.int32,), q.device)
    _tensor(page_table, "page_table", 2, (torch.int32,), q.device)
    _unit_inner(page_table, "page_table")
    if page_table.shape[0] != B:
        raise ValueError("page_table must have one row for each sequence")
    if key_scales is not None:
        _exact(key_scales, "key_scales", (pages, page_size), (torch.float32,), q.device)
    if out is None:
        width = page_table.shape[1] * page_size if width is None else int(width)
        out = torch.empty((B, T, width), dtype=torch.float32, device=q.device)
    else:
        _tensor(out, "out", 3, (torch.float32,), q.device)
        if tuple(out.shape[:2]) != (B, T) or (width is not None and out.shape[2] != width):
            raise ValueError("out must be a tensor [B, T, width]")
        width = out.shape[2]
    _unit_inner(out, "out")
    _no_self_overlap(out, "out")
    if width > page_table.shape[1] * page_size:
        raise ValueError("page_table is too narrow for the width of out")
    a = _ScoresArgs(q=q.data_ptr(), q_seq_stride=q.stride(0), q_token_stride=q.stride(1),
                    q_head_stride=q.stride(2), weights=weights.data_ptr(), keys=keys.data_ptr(),
                    key_page_stride=keys.stride(0), key_token_stride=keys.stride(1),
                    key_scales=_ptr(key_scales), lengths=lengths.data_ptr(), page_table=page_table.data_ptr(),
                    table_stride=page_table.stride(0), table_width=page_table.shape[1], out=out.data_ptr(),
                    out_seq_stride=out.stride(0), out_token_stride=out.stride(1), num_pages=pages,
                    width=width, page_size=page_size, B=B, T=T, H=H, D=D, type=_TYPES[q.dtype])
    _call("sparse_indexer_scores", a, q.get_device(), stream)
    return out


def sparse_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, indices: torch.Tensor,
                     page_table: Optional[torch.Tensor] = None, *,
                     query_positions: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                     first: Optional[torch.Tensor] = None, return_lse: bool = False,
                     out: Optional[torch.Tensor] = None, stream=None):
    """Attention of every query token over its selected entries of a paged cache.

    ``q`` ``[B, T, Hq, D]``; ``k`` ``[pages, page_size, Hkv, D]`` and ``v`` ``[pages, page_size, Hkv,
    Dv]`` of the same type, bfloat16 or float16 (``v`` may be the first ``Dv`` elements of ``k``);
    ``indices`` int32 ``[B, T, K]``, the selected positions, negative where there is none
    (:func:`topk_ragged`), mapped through ``page_table`` int32 ``[B, n]``; without a page table they
    are slots (:func:`topk_paged`).

    ``scale`` (default ``D ** -0.5``) multiplies the products, ``softcap`` caps them by ``softcap *
    tanh(z / softcap)``, ``slopes`` float32 ``[Hq]`` adds ``slopes[h] * (position -
    query_positions[b, t])``. ``query_positions`` int32 ``[B, T]`` hides later positions, ``first``
    int32 ``[B, T]`` earlier ones (a document's start). Returns ``out`` ``[B, T, Hq, Dv]``, with
    ``return_lse`` also the logarithm of the softmax's sum, float32 ``[B, T, Hq]``; a row that sees
    nothing has 0 and ``-inf``."""
    _tensor(q, "q", 4, (torch.bfloat16, torch.float16))
    _unit_inner(q, "q")
    B, T, Hq, D = q.shape
    _tensor(k, "k", 4, (q.dtype,), q.device)
    _tensor(v, "v", 4, (q.dtype,), q.device)
    _unit_inner(k, "k")
    _unit_inner(v, "v")
    pages, page_size, Hkv = k.shape[:3]
    Dv = v.shape[3]
    if k.shape[3] != D or v.shape[:3] != k.shape[:3]:
        raise ValueError("k must be [pages, page_size, Hkv, D] and v [pages, page_size, Hkv, Dv]")
    if Hkv < 1 or Hq % Hkv:
        raise ValueError("the query heads must be a multiple of the key heads")
    _tensor(indices, "indices", 3, (torch.int32,), q.device)
    _exact(indices, "indices", (B, T, indices.shape[2]), (torch.int32,), q.device)
    if page_table is not None:
        _tensor(page_table, "page_table", 2, (torch.int32,), q.device)
        _unit_inner(page_table, "page_table")
        if page_table.shape[0] != B:
            raise ValueError("page_table must have one row for each sequence")
    elif query_positions is not None or first is not None or slopes is not None:
        raise ValueError("slots have no position: query_positions, first and slopes need a page_table")
    if slopes is not None:
        _exact(slopes, "slopes", (Hq,), (torch.float32,), q.device)
        if query_positions is None:
            raise ValueError("slopes need query_positions")
    for t, name in ((query_positions, "query_positions"), (first, "first")):
        if t is not None:
            _exact(t, name, (B, T), (torch.int32,), q.device)
    scale = D ** -0.5 if scale is None else float(scale)
    if not math.isfinite(scale) or not math.isfinite(softcap) or softcap < 0.0:
        raise ValueError("scale and softcap must be finite, softcap not negative")
    if out is None:
        out = torch.empty((B, T, Hq, Dv), dtype=q.dtype, device=q.device)
    else:
        _exact(out, "out", (B, T, Hq, Dv), (q.dtype,), q.device)
        if any(_overlap(out, t) for t in (q, k, v)):
            raise ValueError("out must not overlap q, k or v")
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    a = _AttentionArgs(q=q.data_ptr(), q_seq_stride=q.stride(0), q_token_stride=q.stride(1),
                       q_head_stride=q.stride(2), k=k.data_ptr(), k_page_stride=k.stride(0),
                       k_token_stride=k.stride(1), k_head_stride=k.stride(2), v=v.data_ptr(),
                       v_page_stride=v.stride(0), v_token_stride=v.stride(1), v_head_stride=v.stride(2),
                       indices=indices.data_ptr(), page_table=_ptr(page_table),
                       table_stride=0 if page_table is None else page_table.stride(0),
                       table_width=0 if page_table is None else page_table.shape[1],
                       query_positions=_ptr(query_positions), first=_ptr(first), slopes=_ptr(slopes),
                       out=out.data_ptr(), lse=_ptr(lse), num_pages=pages, page_size=page_size, B=B, T=T,
                       Hq=Hq, Hkv=Hkv, D=D, Dv=Dv, K=indices.shape[2], type=_TYPES[q.dtype], scale=scale,
                       softcap=float(softcap))
    _call("sparse_attention", a, q.get_device(), stream)
    return (out, lse) if return_lse else out
