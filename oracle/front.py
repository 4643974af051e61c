"""The operators in front of the expert layer, written out in float64 from the definitions in
include/mega_moe.h: residual RMS norm with 8-bit output, gate product, choice of experts.

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

from . import codecs as C


def norm_quant(x, residual, weight, eps, recipe):
    """Values before their rounding: h (residual_out), v (normed), the scales (float64; per-32
    recipes also their codes) and v / scale.  Arguments are float arrays [T, H] and [H]."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    T, H = h.shape
    with np.errstate(over="ignore", invalid="ignore"):
        v = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    g = 128 if recipe == 0 else 32
    groups = v.reshape(T, H // g, g)
    r = np.abs(groups).max(axis=2) / C.E4M3_MAX
    code = None
    if recipe == 0:
        sf = r
    else:
        m, e = np.frexp(r)                             # r = m 2^e, m in [0.5, 1)
        code = np.where(r > 0, np.clip(np.where(m == 0.5, e - 1, e) + 127, 0, 254), 0).astype(np.int64)
        sf = np.where(r > 0, C.ue8m0_decode(code), 0.0)
    scaled = np.divide(groups, sf[..., None], out=np.zeros_like(groups), where=sf[..., None] > 0)
    return dict(h=h, v=v, sf=sf, code=code, scaled=scaled.reshape(T, H))


def gate_logits(x, w):
    """The products' sums and the sums of their magnitudes, float64."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def gate_topk(logits, bias, k, score="softmax", num_groups=1, topk_groups=1, group_top=1, num_shared=0, scale=1.0,
              shared_weight=1.0, renorm=False, num_valid=None):
    """topk_idx int32 and topk_w float64 [T, k + num_shared], row by row."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    n = E // num_groups
    b = None if bias is None else np.asarray(bias, dtype=np.float64)
    idx = np.full((T, k + num_shared), -1, dtype=np.int32)
    w = np.zeros((T, k + num_shared))
    valid = T if num_valid is None else min(max(int(num_valid), 0), T)
    for t in range(valid):
        row = np.where(np.isnan(l[t]), -np.inf, l[t])
        counted = row > -np.inf
        candidate = counted.copy()
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-row))
            else:
                top = row.max()
                s = np.where(counted, np.where(row == top, 1.0, np.exp(row - top)), 0.0)
                s = s / s.sum()
        if b is not None:
            candidate &= ~(np.isnan(b) | (b == -np.inf))
            order = group_by = s + b
        else:
            order, group_by = row, (s if group_top == 2 else row)
        if num_groups > 1:
            values = []
            for g in range(num_groups):
                c = sorted((group_by[e] for e in range(g * n, (g + 1) * n) if candidate[e]), reverse=True)[:group_top]
                values.append(sum(c) if c else None)
            kept = sorted((g for g in range(num_groups) if values[g] is not None), key=lambda g: (-values[g], g))
            kept = set(kept[:topk_groups])
            candidate &= np.array([e // n in kept for e in range(E)])
        chosen = sorted((e for e in range(E) if candidate[e]), key=lambda e: (-order[e], e))[:k]
        ws = np.array([s[e] for e in chosen])
        if renorm:
            ws = ws / (ws.sum() + 1e-20)
        idx[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = ws * scale
        idx[t, k:] = np.arange(E, E + num_shared)
        w[t, k:] = shared_weight
    return idx, w
