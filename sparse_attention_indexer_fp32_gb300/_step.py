"""ctypes binding of the operators around the selection (``include/sparse_step.h``).

As in ``_binding``: tensors are checked here, the rest by the library; every
step runs in its CUDA kernels, on the stream given or the current one, and
there is no CPU fallback. The calls record no gradient: tensors that require one
are refused while gradients are recorded, and an ``out`` of the caller's counts as
changed in place.
"""

from __future__ import annotations

import ctypes
import math
import struct
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



# The current device's index and the handle of its current stream, without the
# Python objects around them (torch.cuda's own functions, a microsecond less).
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _raw_stream_slow(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream_slow)


_FORMATS = {_i32: "i", _i64: "q", _f32: "f", _vp: "P"}
_BF16, _FP16, _FP32, _E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
_I32, _I64, _F64 = torch.int32, torch.int64, torch.float64
_ROTARY_TYPES = {_BF16: 0, _FP16: 1, _FP32: 2}
_SCORES_TYPES = {_BF16: 0, _FP16: 1, _E4M3: 3}
_ATTENTION_TYPES = {_BF16: 0, _FP16: 1}
_LAYOUTS = {"half": 0, "interleaved": 1}


class _Call:
    """An entry point of the library. Its arguments are packed into the bytes
    of its C struct in one step: setting the fields of a ctypes Structure one
    by one costs several microseconds of host time a call."""

    def __init__(self, name: str, args):
        self.name, self.fn = name, None
        self.pack = struct.Struct("@" + "".join(_FORMATS[t] for _, t in args._fields_) + "0q").pack

    def __call__(self, index: int, stream, *values) -> None:
        fn = self.fn
        if fn is None:
            lib = _binding.load_library()
            prototype = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, _vp)
            fn = self.fn = prototype(ctypes.cast(getattr(lib, self.name), _vp).value)
        try:
            packed = self.pack(*values)
        except (struct.error, OverflowError) as error:
            raise ValueError(f"{self.name}: an argument is out of range ({error})") from None
        handle = _raw_stream(index) if stream is None else stream.cuda_stream
        if _current_device() == index:
            status = fn(packed, handle)
        else:
            with torch.cuda.device(index):
                status = fn(packed, handle)
        if status != 0:
            message = _binding.load_library().topk_status_string(status).decode()
            raise _binding.TopkError(status, f"{self.name} failed: {message}")


_rotary, _scores, _attention = (_Call("sparse_rotary", _RotaryArgs), _Call("sparse_indexer_scores", _ScoresArgs),
                                _Call("sparse_attention", _AttentionArgs))


def _no_gradient(name: str) -> None:
    """The calls record no backward pass, so they take nothing that would need one."""
    if torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and the call records none: detach it, or call under torch.no_grad()")


# Tells autograd that the caller's tensor has changed, as an in-place operation of torch does.
_written = torch.autograd.graph.increment_version


def _dims(t, name: str, dims: int) -> None:
    raise ValueError(f"{name} must be a {dims}-D tensor")


def _main(t, name: str, dims: int, types):
    """Shape, strides, type code and device of a call's main tensor."""
    try:
        shape, strides, index, code = t.shape, t.stride(), t.get_device(), types.get(t.dtype)
        if t.requires_grad:
            _no_gradient(name)
    except AttributeError:
        _dims(t, name, dims)
    if len(shape) != dims:
        _dims(t, name, dims)
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(str(d) for d in types)}, not {t.dtype}")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return shape, strides, code, index


def _other(t, name: str, dims: int, dtype, index: int):
    """Shape and strides of a further tensor of this type on that device."""
    try:
        shape, strides = t.shape, t.stride()
        if t.requires_grad:
            _no_gradient(name)
    except AttributeError:
        _dims(t, name, dims)
    if len(shape) != dims:
        _dims(t, name, dims)
    if t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the other arguments")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return shape, strides


def _whole(t, name: str, shape, dtype, index: int) -> int:
    """The address of a contiguous tensor of exactly this shape and type."""
    try:
        if t.dtype == dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            if t.requires_grad:
                _no_gradient(name)
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on the device of the other "
                     "arguments")


def _empty(shape, dtype, like, stream):
    """A result's memory, which belongs to the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _span(address: int, shape, strides, size: int):
    """The bytes [start, end) that the elements of a tensor lie within."""
    if 0 in shape:
        return address, address
    return address, address + (sum((n - 1) * s for n, s in zip(shape, strides)) + 1) * size


def _overlap(a, b) -> bool:
    return a[0] < b[1] and b[0] < a[1]


def _no_broadcast(shape, strides, name: str) -> None:
    """An output may not have two of its elements at one address."""
    if 0 in strides and any(s == 0 and n > 1 for n, s in zip(shape, strides)):
        raise ValueError(f"{name} must not be a broadcast tensor")


def rotary_frequencies(rotated: int, base: float = 10000.0, *, scaling: Optional[str] = None,
                       factor: float = 1.0, original_length: int = 4096, fast: float = 32.0,
                       slow: float = 1.0, device="cuda") -> torch.Tensor:
    """Radians per position of each of ``rotated // 2`` pairs, ``base ** (-2 i / rotated)``, float64
    on ``device``, for :func:`rotary`.

    ``scaling`` stretches a context of ``original_length`` positions by ``factor``: ``"linear"``
    divides every frequency by it; ``"base"`` raises the base to ``base * factor ** (rotated /
    (rotated - 2))``, which keeps the fastest pair and divides the slowest by the factor; ``"ramp"``
    keeps pairs that turn more than ``fast`` times within ``original_length`` (the first at least),
    divides those that turn less than ``slow`` times, and blends linearly over the pairs between (the by-parts interpolation of
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
        if base <= 1.0:
            raise ValueError("the ramp needs a base above 1")

        def pair(turns: float) -> float:  # the (fractional) pair that turns so often
            return rotated * math.log(original_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        # either end may lie past the last pair: the ramp is then cut off there
        low, high = max(math.floor(pair(fast)), 0), max(math.ceil(pair(slow)), 0)
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
    of the call with the same arguments. ``out`` may be ``x`` (in place); the addresses of any other
    ``out`` lie wholly before or behind those of ``x``. With ``slots`` (int32
    ``[T]``), ``out`` is a paged cache ``[pages, page_size, H, D]`` and token ``t`` is written at slot
    ``slots[t]`` (negative or past the cache: not written). Returns ``out``."""
    shape, xs, code, index = _main(x, "x", 3, _ROTARY_TYPES)
    T, H, D = shape
    dtype = x.dtype
    wide = isinstance(positions, torch.Tensor) and positions.dtype == _I64
    pos = _whole(positions, "positions", (T,), _I64 if wide else _I32, index)
    pairs = frequencies.numel() if isinstance(frequencies, torch.Tensor) else 0
    freq = _whole(frequencies, "frequencies", (pairs,), _F64, index)
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    to, pages, page_size, page_stride = 0, 0, 0, 0
    address, given = x.data_ptr(), out is not None
    if slots is not None:
        if out is None:
            raise ValueError("slots need the cache as out")
        os, ot = _other(out, "out", 4, dtype, index)
        if os[2:] != (H, D):
            raise ValueError("out must be a cache [pages, page_size, H, D]")
        to = _whole(slots, "slots", (T,), _I32, index)
        pages, page_size, page_stride = os[0], os[1], ot[0]
    elif out is not None:
        os, ot = _other(out, "out", 3, dtype, index)
        if os != shape:
            raise ValueError("out must have the shape of x")
    if out is None:
        out = _empty(shape, dtype, x, stream)
        target, ot = out.data_ptr(), out.stride()
    else:
        target = out.data_ptr()
        _no_broadcast(os, ot, "out")
        if slots is not None or target != address or any(n > 1 and u != v for n, u, v in zip(shape, xs, ot)):
            size = 4 if code == 2 else 2
            if _overlap(_span(address, shape, xs, size), _span(target, os, ot, size)):
                raise ValueError("out must be x itself or not overlap it")
    _rotary(index, stream, address, xs[0], xs[1], target, page_stride, ot[-3], ot[-2], pos, freq, to, pages, page_size,
            T, H, D, 2 * pairs, int(offset), _LAYOUTS[layout], code, wide, bool(inverse), scale)
    if given:
        _written(out)
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
    shape, qs, code, index = _main(q, "q", 4, _SCORES_TYPES)
    B, T, H, D = shape
    w = _whole(weights, "weights", (B, T, H), _FP32, index)
    ks, kt = _other(keys, "keys", 3, q.dtype, index)
    pages, page_size, entry = ks
    if entry != D:
        raise ValueError("keys must have the head size of q")
    n = _whole(lengths, "lengths", (B, T), _I32, index)
    ps, pt = _other(page_table, "page_table", 2, _I32, index)
    if ps[0] != B:
        raise ValueError("page_table must have one row for each sequence")
    given = out is not None
    scales = 0 if key_scales is None else _whole(key_scales, "key_scales", (pages, page_size), _FP32, index)
    if out is None:
        width = ps[1] * page_size if width is None else int(width)
        out = _empty((B, T, width), _FP32, q, stream)
        ot = out.stride()
    else:
        os, ot = _other(out, "out", 3, _FP32, index)
        if os[:2] != (B, T) or (width is not None and os[2] != width):
            raise ValueError("out must be a tensor [B, T, width]")
        width = os[2]
        _no_broadcast(os, ot, "out")
    if width > ps[1] * page_size:
        raise ValueError("page_table is too narrow for the width of out")
    _scores(index, stream, q.data_ptr(), qs[0], qs[1], qs[2], w, keys.data_ptr(), kt[0], kt[1], scales, n,
            page_table.data_ptr(), pt[0], ps[1], out.data_ptr(), ot[0], ot[1], pages, width, page_size, B, T, H, D, code)
    if given:
        _written(out)
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
    shape, qs, code, index = _main(q, "q", 4, _ATTENTION_TYPES)
    B, T, Hq, D = shape
    dtype = q.dtype
    ks, kt = _other(k, "k", 4, dtype, index)
    vs, vt = _other(v, "v", 4, dtype, index)
    pages, page_size, Hkv = ks[:3]
    Dv = vs[3]
    if ks[3] != D or vs[:3] != ks[:3]:
        raise ValueError("k must be [pages, page_size, Hkv, D] and v [pages, page_size, Hkv, Dv]")
    if Hkv < 1 or Hq % Hkv:
        raise ValueError("the query heads must be a multiple of the key heads")
    K = indices.shape[-1] if isinstance(indices, torch.Tensor) and indices.dim() else 0
    idx = _whole(indices, "indices", (B, T, K), _I32, index)
    table, pt, width = 0, 0, 0
    if page_table is not None:
        ps, strides = _other(page_table, "page_table", 2, _I32, index)
        if ps[0] != B:
            raise ValueError("page_table must have one row for each sequence")
        table, pt, width = page_table.data_ptr(), strides[0], ps[1]
    elif query_positions is not None or first is not None or slopes is not None:
        raise ValueError("slots have no position: query_positions, first and slopes need a page_table")
    if slopes is not None and query_positions is None:
        raise ValueError("slopes need query_positions")
    bias = 0 if slopes is None else _whole(slopes, "slopes", (Hq,), _FP32, index)
    qp = 0 if query_positions is None else _whole(query_positions, "query_positions", (B, T), _I32, index)
    begin = 0 if first is None else _whole(first, "first", (B, T), _I32, index)
    scale = D ** -0.5 if scale is None else float(scale)
    if not math.isfinite(scale) or not math.isfinite(softcap) or softcap < 0.0:
        raise ValueError("scale and softcap must be finite, softcap not negative")
    if 0.0 < softcap < 2.0 ** -149:
        raise ValueError("softcap must be 0 or a positive float32")
    given = out is not None
    at_q, at_k, at_v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    if out is None:
        out = _empty((B, T, Hq, Dv), dtype, q, stream)
        target = out.data_ptr()
    else:
        target = _whole(out, "out", (B, T, Hq, Dv), dtype, index)
        mine = (target, target + 2 * B * T * Hq * Dv)
        if _overlap(mine, _span(at_q, shape, qs, 2)) or _overlap(mine, _span(at_k, ks, kt, 2)) \
                or _overlap(mine, _span(at_v, vs, vt, 2)):
            raise ValueError("out must not overlap q, k or v")
    lse = _empty((B, T, Hq), _FP32, q, stream) if return_lse else None
    _attention(index, stream, at_q, qs[0], qs[1], qs[2], at_k, kt[0], kt[1], kt[2], at_v, vt[0], vt[1], vt[2], idx, table,
               pt, width, qp, begin, bias, target, 0 if lse is None else lse.data_ptr(), pages, page_size, B, T, Hq, Hkv,
               D, Dv, K, code, scale, softcap)
    if given:
        _written(out)
    return (out, lse) if return_lse else out
