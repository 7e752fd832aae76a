"""The operators around the selection in 64 bits, as their formulas (numpy,
row by row), each with a bound on how far a correct FP32 computation can be
from it.

Bounds. Products of 16- and 8-bit values are exact in FP32. A sum of n FP32
terms in any order is off by at most n 2^-24 of the sum of their magnitudes
when every addition rounds to nearest, n 2^-23 when it truncates (tensor
cores); the bounds take the second. A result rounded to a type of eps is off by
eps / 2 of itself.
"""

from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -23


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def np64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def npi(t):
    return None if t is None else t.detach().cpu().numpy().astype(np.int64)


def rotary(x, positions, frequencies, layout, offset, scale, inverse):
    """(result, bound). The trigonometric functions are good to 2 ulp (of 1),
    the angle to 2^-31 turns, and three FP32 roundings follow: 16 U of the
    pair's length covers them."""
    dtype, x, f = x.dtype, np64(x), np64(frequencies)
    R = 2 * len(f)
    a = npi(positions).astype(np.longdouble)[:, None] * f.astype(np.longdouble)
    c, s = (np.asarray(g(a), dtype=np.float64)[:, None, :] * scale for g in (np.cos, np.sin))
    if inverse:
        s = -s
    y, err = x.copy(), np.zeros_like(x)
    one = slice(offset, offset + R // 2) if layout == "half" else slice(offset, offset + R, 2)
    two = slice(offset + R // 2, offset + R) if layout == "half" else slice(offset + 1, offset + R, 2)
    u, v = x[..., one], x[..., two]
    y[..., one], y[..., two] = u * c - v * s, v * c + u * s
    length = abs(scale) * np.hypot(u, v) * 16 * U
    for part in (one, two):
        err[..., part] = half_step(dtype) * np.abs(y[..., part]) + length * (1 + half_step(dtype))
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # results under the smallest normal value
    err[..., offset:offset + R] += tiny
    return y, err


def slots_of(table_row, positions, page_size, num_pages):
    """Slots of positions, -1 where the page lies outside the table or the cache."""
    out = np.full(len(positions), -1, dtype=np.int64)
    for i, p in enumerate(positions):
        if p < 0 or (table_row is not None and p // page_size >= len(table_row)):
            continue
        page = p // page_size if table_row is None else table_row[p // page_size]
        if 0 <= page < num_pages:
            out[i] = page * page_size + p % page_size
    return out


def scores(q, weights, keys, lengths, table, key_scales, width):
    """(result with NaN where nothing is written, bound)."""
    B, T, H, D = q.shape
    pages, ps = keys.shape[:2]
    q, w, lengths, table = np64(q.float()), np64(weights), npi(lengths), npi(table)
    flat = np64(keys.float()).reshape(pages * ps, D)
    ks = None if key_scales is None else np64(key_scales).reshape(-1)
    out, err = np.full((B, T, width), np.nan), np.zeros((B, T, width))
    for b in range(B):
        sl = slots_of(table[b], np.arange(width), ps, pages)
        k = flat[np.maximum(sl, 0)]
        scale = np.ones(width) if ks is None else ks[np.maximum(sl, 0)]
        for t in range(T):
            n = min(max(lengths[b, t], 0), width)
            with np.errstate(invalid="ignore", over="ignore"):
                dots = q[b, t] @ k.T
                got = (w[b, t] @ np.where(dots > 0, dots, np.where(np.isnan(dots), np.nan, 0.0))) * scale
                mass = (np.abs(w[b, t]) @ (np.abs(q[b, t]) @ np.abs(k).T)) * np.abs(scale)
            got = np.where(sl < 0, -np.inf, got)
            out[b, t, :n], err[b, t, :n] = got[:n], ((D + H + 8) * U * mass)[:n]
    return out, err


def attention(q, k, v, indices, table, query_positions, scale, softcap, slopes, first):
    """(out, its bound, lse, its bound). An error dz of a logit is a relative
    error dz of its weight; with it come the rounding of the weight to the
    type of v (half a step), the sum's and the output's own rounding."""
    B, T, Hq, D = q.shape
    pages, ps, Hkv, Dv = v.shape
    K = indices.shape[2]
    hs = half_step(v.dtype)
    tiny = torch.finfo(v.dtype).tiny * torch.finfo(v.dtype).eps
    q, idx = np64(q), npi(indices)
    kf, vf = np64(k).reshape(pages * ps, Hkv, D), np64(v).reshape(pages * ps, Hkv, Dv)
    table, qp, first, slopes = npi(table), npi(query_positions), npi(first), np64(slopes)
    out, oerr = np.zeros((B, T, Hq, Dv)), np.zeros((B, T, Hq, Dv))
    lse, lerr = np.full((B, T, Hq), -np.inf), np.zeros((B, T, Hq))
    for b in range(B):
        for t in range(T):
            pos = idx[b, t]
            sl = slots_of(None if table is None else table[b], pos, ps, pages) if pages * ps else np.full(K, -1)
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
                kk, vv = kf[sl, g], vf[sl, g]
                z = kk @ q[b, t, h] * scale
                dz = (D + 4) * U * abs(scale) * (np.abs(kk) @ np.abs(q[b, t, h])) + 4 * U * np.abs(z)
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                    dz = dz + 8 * U * softcap
                if slopes is not None:
                    away = slopes[h] * (pos - qp[b, t])
                    z = z + away
                    dz = dz + 4 * U * (np.abs(away) + np.abs(z))
                top = z.max()
                e = np.exp(z - top)
                dz = dz + 4 * U * np.abs(z - top) + 8 * U
                p, total = e / e.sum(), e.sum()
                out[b, t, h] = p @ vv
                mean_dz = p @ dz + (len(sl) + 8) * U
                # weights under the type's smallest value are lost whole: each adds at most it, relative to the largest
                lost = tiny * np.abs(vv).sum(axis=0) / total
                oerr[b, t, h] = ((p * (hs + dz + mean_dz)) @ np.abs(vv)) * 1.01 + lost + hs * np.abs(out[b, t, h]) * 1.01 + tiny
                lse[b, t, h] = np.log(total) + top
                lerr[b, t, h] = mean_dz + 4 * U * (abs(top) + abs(lse[b, t, h]))
    return out, oerr, lse, lerr


def assert_near(got, want, bound, what="") -> None:
    """Every value within its bound; NaN and infinities in the same places."""
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (got.shape, want.shape)
    same = np.isfinite(want) == np.isfinite(got)
    assert same.all(), f"{what}: {np.argwhere(~same)[:5].tolist()} finite on one side only"
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), f"{what}: infinities or NaN differ"
    over = np.abs(got[~odd] - want[~odd]) - bound[~odd]
    if over.size and over.max() > 0:
        i = np.argwhere(~odd)[int(over.argmax())]
        raise AssertionError(f"{what}: at {i.tolist()} {got[tuple(i)]} for {want[tuple(i)]}, bound {bound[tuple(i)]}"
                             f" ({int((over > 0).sum())} of {over.size} over)")
