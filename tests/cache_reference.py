"""The operators of a paged cache in 8 bits, as their formulas in 64 bits (numpy), with bounds counted from
the roundings. What holds for products, sums and the cache's own layout is in ``step_reference``."""

from __future__ import annotations

import numpy as np
import torch

import step_reference as R

E4M3 = torch.float8_e4m3fn
CODES = np.arange(256, dtype=np.uint8)
VALUES = torch.from_numpy(CODES.copy()).view(E4M3).double().numpy()  # of every code


def power_for(most: float) -> float:
    """The smallest power of two, 2^-126 at least, with most <= 448 times it."""
    s = 2.0 ** -126
    while most > 448.0 * s:
        s *= 2.0
    return s


def round_e4m3(x):
    """To nearest, ties to even, past 448 to 448, NaN and infinities to NaN; float64 in and out."""
    x = np.asarray(x, dtype=np.float64)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -30))), -6.0) - 3.0)
    with np.errstate(invalid="ignore"):
        y = np.clip(np.round(x / step) * step, -448.0, 448.0)  # numpy rounds ties to even
    return np.where(np.isfinite(x), y, np.nan)


def append(x, positions, frequencies, cache, scales, slots, block, layout="half", offset=0, scale=1.0):
    """(cache, bound, scales) after one side of the call, the cache as float64 values of its codes (or of its
    type). `frequencies` None: not rotated. A token's number is off by the rotation's bound and a rounding; one
    that is held stays as it is or is rounded again exactly."""
    dtype = cache.dtype
    pages, page_size = cache.shape[:2]
    got = R.np64(cache.float() if dtype == E4M3 else cache).copy()
    flat = got.reshape(pages * page_size, *got.shape[2:])
    err = np.zeros_like(flat)
    slots = R.npi(slots)
    kept = [t for t in range(len(slots)) if 0 <= slots[t] < len(flat)]
    if frequencies is None:
        y, far = R.np64(x), np.zeros(x.shape)
        size = np.abs(y)
    else:
        wide, far = R.rotary(x.float(), positions, frequencies, layout, offset, scale, False)
        y, half = wide, frequencies.numel()
        one = slice(offset, offset + half) if layout == "half" else slice(offset, offset + 2 * half, 2)
        two = slice(offset + half, offset + 2 * half) if layout == "half" else slice(offset + 1, offset + 2 * half, 2)
        size = np.abs(R.np64(x))
        size[..., one] = size[..., two] = (size[..., one] + size[..., two]) * abs(scale)
        # the special function unit's 2^-21 instead of 2 ulp, for each of a pair's two products
        far[..., offset:offset + 2 * half] += 2.0 ** -20 * size[..., offset:offset + 2 * half]
    if dtype != E4M3:
        tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
        for t in kept:
            flat[slots[t]] = y[t]
            err[slots[t]] = far[t] + R.half_step(dtype) * (np.abs(y[t]) + far[t]) + tiny
            same = np.ones(y.shape[-1], dtype=bool)
            if frequencies is not None:
                same[offset:offset + 2 * half] = False
            err[slots[t]][:, same] = 0.0
        return got, err.reshape(got.shape), None
    new = R.np64(scales).copy()
    units = new.reshape(-1, new.shape[-1])
    for b in sorted({slots[t] // block for t in kept}):
        mine = [t for t in kept if slots[t] // block == b]
        first = min(slots[t] % block for t in mine)
        for h in range(units.shape[1]):
            sizes = size[mine, h]
            sizes = sizes[np.isfinite(sizes)]
            need = power_for(sizes.max() if sizes.size else 0.0)
            old = units[b, h]
            units[b, h] = need if first == 0 else max(old, need)
            if first and units[b, h] != old:
                held = slice(b * block, b * block + first)
                flat[held, h] = round_e4m3(flat[held, h] * (old / units[b, h]))
    for t in kept:
        unit = units[slots[t] // block][:, None]
        exact, off = y[t] / unit, far[t] / unit
        flat[slots[t]] = np.where(np.isfinite(exact), np.clip(exact, -448.0, 448.0), np.nan)
        err[slots[t]] = off + np.maximum((np.abs(exact) + off) * 2.0 ** -4, 2.0 ** -10) + 2.0 ** -22 * np.abs(exact)
    return got, err.reshape(got.shape), new


def entries(cache, scales):
    """What the entries of a cache in 8 bits stand for, float64 [pages, page_size, heads, size], and their scales."""
    page_size, blocks = cache.shape[1], scales.shape[1]
    units = np.repeat(R.np64(scales), page_size // blocks, axis=1)[..., None]
    return R.np64(cache.float()), units


def attention(q, k, v, k_scales, v_scales, indices, table, query_positions, scale, softcap=0.0, slopes=None, first=None):
    """(out, its bound, lse, its bound). As step_reference.attention, with what this form rounds: a query's terms
    end at half a step of 2^-20 (bf16) or 2^-24 of its largest element; a weight is rounded to fp16 and to 9 bits
    (bf16) or to fp16, and ends at half a step of 2^-16 or 2^-20 of the largest weight, each times its value's scale."""
    B, T, Hq, D = q.shape
    pages, ps, Hkv, Dv = v.shape
    q_type, U, three = q.dtype, R.U, q.dtype == torch.float16
    rounded = 2.0 ** -11 if three else 2.0 ** -9 + 2.0 ** -11
    query_end, weight_end = (2.0 ** -25, 2.0 ** -21) if three else (2.0 ** -21, 2.0 ** -17)
    hs, tiny = R.half_step(q.dtype), torch.finfo(q.dtype).tiny * torch.finfo(q.dtype).eps
    (kf, ku), (vf, vu) = entries(k, k_scales), entries(v, v_scales)
    kf, ku, vf, vu = kf.reshape(-1, Hkv, D), ku.reshape(-1, Hkv), vf.reshape(-1, Hkv, Dv), vu.reshape(-1, Hkv)
    q, idx, table, qp, first, slopes = R.np64(q), R.npi(indices), R.npi(table), R.npi(query_positions), R.npi(first), R.np64(slopes)
    out, oerr = np.zeros((B, T, Hq, Dv)), np.zeros((B, T, Hq, Dv))
    lse, lerr = np.full((B, T, Hq), -np.inf), np.zeros((B, T, Hq))
    for b in range(B):
        for t in range(T):
            pos = idx[b, t]
            sl = R.slots_of(None if table is None else table[b], pos, ps, pages) if pages * ps else np.full(len(pos), -1)
            ok = sl >= 0
            if qp is not None:
                ok &= pos <= qp[b, t]
            if first is not None:
                ok &= pos >= first[b, t]
            sl, pos = sl[ok], pos[ok]
            if not len(sl):
                continue
            for h in range(Hq):
                g = h // (Hq // Hkv)
                x, kk, vv, vs = q[b, t, h], kf[sl, g] * ku[sl, g, None], vf[sl, g], vu[sl, g]
                z = kk @ x * scale
                dz = abs(scale) * ((D + 8) * U * (np.abs(kk) @ np.abs(x)) + query_end * np.abs(x).max() * np.abs(kk).sum(1))
                dz = dz + 6 * U * np.abs(z)
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                    dz = dz + 8 * U * np.abs(z)
                if slopes is not None:
                    away = slopes[h] * (pos - qp[b, t])
                    z = z + away
                    dz = dz + 4 * U * (np.abs(away) + np.abs(z))
                top = z.max()
                e = np.exp(z - top)
                dz = dz + 4 * U * np.abs(z - top) + 8 * U
                p, total = e / e.sum(), e.sum()
                w = p * vs
                out[b, t, h] = w @ vv
                mean_dz = p @ dz + (len(sl) + 8) * U
                end = weight_end * (p * np.maximum(np.abs(vs), 2.0 ** -60)).max()
                oerr[b, t, h] = ((np.abs(w) * (rounded + dz + mean_dz) + end) @ np.abs(vv)) * 1.01 \
                    + hs * np.abs(out[b, t, h]) * 1.01 + tiny
                lse[b, t, h] = np.log(total) + top
                lerr[b, t, h] = mean_dz + 4 * U * (abs(top) + abs(lse[b, t, h]))
    with np.errstate(invalid="ignore"):  # a result past the type's largest number rounds to infinity
        out = np.where(np.abs(out) > torch.finfo(q_type).max * (1 + 2 * hs), np.copysign(np.inf, out), out)
    return out, oerr, lse, lerr
