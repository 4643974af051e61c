"""The layer in parts, written out in float64 from the definitions in include/mega_moe.h: tokens sorted by expert and
back with its gradient, the 8-bit product by group, the activation with its 8-bit output and its gradient.

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

from . import codecs as C


def sort_plan(topk_idx, E):
    """expert_offset [E + 1], pool_src [n] and pair_pos [T, k] of the n pairs with an id in [0, E)."""
    flat = np.asarray(topk_idx).reshape(-1).astype(np.int64)
    pairs = np.flatnonzero((flat >= 0) & (flat < E))
    src = pairs[np.lexsort((pairs, flat[pairs]))]
    pos = np.full(flat.size, -1, dtype=np.int32)
    pos[src] = np.arange(src.size)
    offset = np.concatenate([[0], np.cumsum(np.bincount(flat[pairs], minlength=E))])
    return offset.astype(np.int32), src.astype(np.int32), pos.reshape(np.shape(topk_idx))


def _with_place(pos, j, num_rows):
    at = np.asarray(pos)[:, j].astype(np.int64)
    t = np.flatnonzero((at >= 0) & (at < num_rows))
    return t, at[t]


def unsort(rows, pos, w=None):
    """y and the sums of the terms' magnitudes."""
    rows = np.asarray(rows, dtype=np.float64)
    y, mag = np.zeros((len(pos), rows.shape[1])), np.zeros((len(pos), rows.shape[1]))
    for j in range(np.shape(pos)[1]):
        t, r = _with_place(pos, j, len(rows))
        term = rows[r] if w is None else rows[r] * np.asarray(w, dtype=np.float64)[t, j, None]
        y[t] += term
        mag[t] += np.abs(term)
    return y, mag


def unsort_backward(dy, rows, pos, w=None):
    """d_rows (NaN at places without a pair), d_w and the sums of the magnitudes of d_w's terms."""
    dy, rows = np.asarray(dy, dtype=np.float64), np.asarray(rows, dtype=np.float64)
    d_rows, d_w, mag = np.full(rows.shape, np.nan), np.zeros(np.shape(pos)), np.zeros(np.shape(pos))
    for j in range(np.shape(pos)[1]):
        t, r = _with_place(pos, j, len(rows))
        d_rows[r] = dy[t] if w is None else dy[t] * np.asarray(w, dtype=np.float64)[t, j, None]
        terms = rows[r] * dy[t]
        d_w[t, j], mag[t, j] = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    return d_rows, d_w, mag


def block_product(x, x_sf, w, w_sf, offset=None):
    """y (NaN outside the groups) and the sums of the magnitudes of its terms; x [M, K] and w [G, N, K] as E4M3 codes."""
    M, K = x.shape
    G, N, _ = w.shape
    y, mag = np.full((M, N), np.nan), np.zeros((M, N))
    ends = [0, M] if offset is None else offset
    for g in range(G):
        lo = min(max(int(ends[g]), 0), M)
        hi = min(max(int(ends[g + 1]), lo), M)
        if lo == hi:
            continue
        xd = C.e4m3_decode(x[lo:hi]) * np.repeat(np.asarray(x_sf[lo:hi], dtype=np.float64), 128, axis=1)
        sf = np.repeat(np.repeat(np.asarray(w_sf[g], dtype=np.float64), 128, axis=0)[:N], 128, axis=1)
        wd = C.e4m3_decode(w[g]) * sf
        y[lo:hi], mag[lo:hi] = xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    return y, mag


def activation(x, act="swiglu", clamp=0.0, inputs=False):
    """v [M, I]."""
    x = np.asarray(x, dtype=np.float64)
    if act == "none":
        return x
    g, u = np.split(x, 2, axis=1)
    if clamp and inputs:
        g, u = np.clip(g, -clamp, clamp), np.clip(u, -clamp, clamp)
    with np.errstate(over="ignore", invalid="ignore"):
        v = g / (1.0 + np.exp(-g)) * u
    return np.clip(v, -clamp, clamp) if clamp and not inputs else v


def scales(v, recipe):
    """The scales of v's groups (float64), and the UE8M0 codes of the per-32 recipes."""
    g = 128 if recipe == 0 else 32
    r = np.abs(v).reshape(len(v), -1, g).max(axis=2) / C.E4M3_MAX
    if recipe == 0:
        return r, None
    m, e = np.frexp(r)                                 # r = m 2^e, m in [0.5, 1)
    code = np.where(r > 0, np.clip(np.where(m == 0.5, e - 1, e) + 127, 0, 254), 0).astype(np.int64)
    return np.ldexp(1.0, code - 127), code


def act_backward(x, d, clamp=0.0, inputs=False):
    """d_x [M, 2I], and what its rounding errors are relative to (the terms before they cancel)."""
    x, d = np.asarray(x, dtype=np.float64), np.asarray(d, dtype=np.float64)
    g0, u0 = np.split(x, 2, axis=1)
    g, u = (np.clip(g0, -clamp, clamp), np.clip(u0, -clamp, clamp)) if clamp and inputs else (g0, u0)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
        rest = 1.0 / (1.0 + np.exp(g))
    d_g, d_u = d * u * s * (1 + g * rest), d * g * s
    mag = np.abs(d * u * s) * (1 + np.abs(g * rest))
    if clamp and not inputs:                           # selected: the dropped terms may not be finite
        d_g, d_u, mag = (np.where(np.abs(g * s * u) > clamp, 0.0, v) for v in (d_g, d_u, mag))
    if clamp and inputs:
        d_g, mag = (np.where(np.abs(g0) > clamp, 0.0, v) for v in (d_g, mag))
        d_u = np.where(np.abs(u0) > clamp, 0.0, d_u)
    return np.concatenate([d_g, d_u], axis=1), np.concatenate([mag, np.abs(d_u)], axis=1)
