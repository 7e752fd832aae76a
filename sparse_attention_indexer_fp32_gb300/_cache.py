"""ctypes binding of the operators of a paged cache in 8 bits
(``include/sparse_cache.h``), by the same rules as ``_step``."""

from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from ._step import (_E4M3, _F64, _I32, _I64, _LAYOUTS, _ROTARY_TYPES, _Call, _main, _no_broadcast, _other, _scales_of,
                    _whole, _written)

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class _AppendArgs(ctypes.Structure):
    _fields_ = [("k", _vp), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v", _vp), ("v_token_stride", _i64), ("v_head_stride", _i64),
                ("k_cache", _vp), ("k_cache_page_stride", _i64), ("k_cache_token_stride", _i64),
                ("k_cache_head_stride", _i64),
                ("v_cache", _vp), ("v_cache_page_stride", _i64), ("v_cache_token_stride", _i64),
                ("v_cache_head_stride", _i64),
                ("k_scales", _vp), ("v_scales", _vp), ("positions", _vp), ("frequencies", _vp), ("slots", _vp),
                ("num_pages", _i64), ("page_size", _i32), ("blocks", _i32), ("T", _i32), ("H", _i32), ("D", _i32),
                ("Dv", _i32), ("rotated", _i32), ("offset", _i32), ("layout", _i32), ("type", _i32),
                ("cache_type", _i32), ("positions_64", _i32), ("scale", _f32)]


_append = _Call("sparse_append", _AppendArgs)


def _entries(cache, name: str, like, heads: int, size: int, index: int):
    """Shape, strides and type of a cache of these heads, its entries in 8 bits or of the type of `like`."""
    held = cache.dtype if isinstance(cache, torch.Tensor) else None
    if held != _E4M3 and held != like:
        raise ValueError(f"{name} must be a 4-D tensor of {like} or {_E4M3}")
    shape, strides = _other(cache, name, 4, held, index)
    if shape[2] != heads or shape[3] != size:
        raise ValueError(f"{name} must be [pages, page_size, {heads}, {size}]")
    _no_broadcast(shape, strides, name)
    return shape, strides, held


def _end(address: int, shape, strides, size: int) -> int:
    """The address behind the last element of a tensor of three or four dimensions, `address` if it has none."""
    if 0 in shape:
        return address
    last = (shape[0] - 1) * strides[0] + (shape[1] - 1) * strides[1] + (shape[2] - 1) * strides[2] + 1
    return address + (last + (shape[3] - 1) * strides[3] if len(shape) == 4 else last) * size


def cache_append(k: torch.Tensor, v: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                 frequencies: Optional[torch.Tensor], k_cache: torch.Tensor, v_cache: Optional[torch.Tensor],
                 slots: torch.Tensor, *, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None, layout: str = "half", offset: int = 0, scale: float = 1.0,
                 stream=None) -> None:
    """Keys, rotated as by :func:`rotary`, and values into paged caches of their own type or in 8 bits.

    ``k`` bfloat16, float16 or float32 ``[T, H, D]`` and ``v`` ``[T, H, Dv]`` of the same type (any
    strides, unit in the last dimension; ``None``, with ``v_cache``, for keys alone); ``positions`` int32 or
    int64 ``[T]`` and ``frequencies`` float64 (:func:`rotary_frequencies`; ``None``, then ``positions`` may be
    ``None`` too, for keys that are not rotated); ``layout``, ``offset`` and ``scale`` as in :func:`rotary`.
    Token ``t`` is written at slot ``slots[t]`` (int32; negative or past the cache: not written) of
    ``k_cache`` ``[pages, page_size, H, D]`` and ``v_cache`` ``[pages, page_size, H, Dv]``.

    Caches in float8_e4m3fn hold entries in units of ``k_scales`` and ``v_scales``, float32 ``[pages, blocks,
    H]``: the ``page_size // blocks`` entries of a block share one for each head. Tokens may come in any order,
    each at a slot of its own (fastest with those of a block one behind the other). A block that a call begins
    at its first place gets the smallest power of two that holds the call's tokens; one that is continued keeps
    its scale while that holds them, otherwise the scale grows and the entries before are rounded again (places
    behind the call's first one count as empty, and so does a block whose scale is 0). ``[pages, page_size, 1]``
    for one head is what :func:`indexer_scores` takes as ``key_scales``; :func:`sparse_attention` reads any."""
    shape, xs, code, index = _main(k, "k", 3, _ROTARY_TYPES)
    T, H, D = shape
    dtype = k.dtype
    to = _whole(slots, "slots", (T,), _I32, index)
    ks, kt, held = _entries(k_cache, "k_cache", dtype, H, D, index)
    pages, page_size = ks[0], ks[1]
    eight = held == _E4M3
    pos, freq, pairs, wide = 0, 0, 0, False
    if frequencies is not None:
        pairs = frequencies.numel() if isinstance(frequencies, torch.Tensor) else 0
        freq = _whole(frequencies, "frequencies", (pairs,), _F64, index)
        wide = isinstance(positions, torch.Tensor) and positions.dtype == _I64
        pos = _whole(positions, "positions", (T,), _I64 if wide else _I32, index)
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    Dv, vx, vt, at_v, to_v = 0, (0, 0), (0, 0, 0), 0, 0
    bytes_in = 4 if code == 2 else 2
    size = 1 if eight else bytes_in
    at_k, to_k = k.data_ptr(), k_cache.data_ptr()
    end_k, end_keys = _end(at_k, shape, xs, bytes_in), _end(to_k, ks, kt, size)
    if at_k < end_keys and to_k < end_k:
        raise ValueError("k_cache must not overlap k")
    if v is not None:
        vs, vx = _other(v, "v", 3, dtype, index)
        if vs[0] != T or vs[1] != H:
            raise ValueError("v must be [T, H, Dv]")
        Dv = vs[2]
        cs, vt, other = _entries(v_cache, "v_cache", dtype, H, Dv, index)
        if cs[0] != pages or cs[1] != page_size or other != held:
            raise ValueError("v_cache must have the pages and the type of k_cache")
        at_v, to_v = v.data_ptr(), v_cache.data_ptr()
        end_v, end_values = _end(at_v, vs, vx, bytes_in), _end(to_v, cs, vt, size)
        if at_v < end_keys and to_k < end_v or at_v < end_values and to_v < end_v or at_k < end_values and to_v < end_k:
            raise ValueError("the caches must not overlap k or v")
        if to_k < end_values and to_v < end_keys and _meet(ks, kt, vt, Dv, to_v - to_k, size):
            raise ValueError("v_cache must not overlap k_cache")
    units_k, units_v, blocks = 0, 0, 0
    if eight:
        units_k, blocks = _scales_of(k_scales, "k_scales", pages, page_size, H, index)
        if v is not None:
            units_v, other = _scales_of(v_scales, "v_scales", pages, page_size, H, index)
            if other != blocks:
                raise ValueError("v_scales must have the blocks of k_scales")
            if units_v == units_k and pages * H > 0:
                raise ValueError("v_scales must not be k_scales: each cache has its own")
        size_of_scales = 4 * pages * blocks * H
        spans = [(at_k, end_k), (to_k, end_keys), (to, to + 4 * T)]
        if freq:
            spans += (pos, pos + (8 if wide else 4) * T), (freq, freq + 8 * pairs)
        if v is not None:
            spans += (at_v, end_v), (to_v, end_values)
            if _clash(units_v, size_of_scales, spans):
                raise ValueError("v_scales must not overlap any other tensor of the call")
            spans.append((units_v, units_v + size_of_scales))
        if _clash(units_k, size_of_scales, spans):
            raise ValueError("k_scales must not overlap any other tensor of the call")
    elif k_scales is not None or v_scales is not None:
        raise ValueError("only caches in float8_e4m3fn have scales")
    _append(index, stream, at_k, xs[0], xs[1], at_v, vx[0], vx[1], to_k, kt[0], kt[1], kt[2], to_v, vt[0], vt[1], vt[2],
            units_k, units_v, pos, freq, to, pages, page_size, blocks, T, H, D, Dv, 2 * pairs, int(offset),
            _LAYOUTS[layout], code, 3 if eight else code, wide, scale)
    _written([t for t in (k_cache, v_cache, k_scales, v_scales) if t is not None])


def _clash(begin: int, size: int, spans) -> bool:
    """Whether `size` bytes from `begin` overlap one of the spans [start, end)."""
    end = begin + size
    for start, stop in spans:
        if start < end and begin < stop and start < stop:
            return size > 0
    return False


def _meet(shape, strides, others, second: int, gap: int, size: int) -> bool:
    """Whether two caches of these pages and heads may share an element, the second one's entries `second`
    elements long and its start `gap` bytes behind the first one's. Parts of one tensor do not: they have its
    strides, each past what the smaller ones reach, and lie side by side in its pages, tokens or entries. Any
    other two whose addresses mix may."""
    if gap % size or any(n > 1 and s != t for n, s, t in zip(shape[:3], strides, others)):
        return True
    dims, reach = [], max(shape[3], second) - 1  # how far two elements lie apart in the smaller dimensions
    for step, n in sorted((s, n) for n, s in zip(shape[:3], strides) if n > 1):
        if step <= reach:
            return True
        dims.append((step, n))
        reach += step * (n - 1)

    def meet(gap, dims):
        if not dims:
            return -second < gap < shape[3]
        step, n = dims[-1]  # the smaller ones reach less than a step: two places at most
        return any(meet(gap - d * step, dims[:-1]) for d in (gap // step, gap // step + 1) if -n < d < n)

    return meet(gap // size, dims)
