"""Plain fp64 reference of the 8-bit integer side of a layer: norm, activation,
products of 8-bit rows, router and experts.  Written from the definitions, one
row or one expert at a time; shares nothing with the HIP path."""
from __future__ import annotations

import numpy as np


def add_rmsnorm(x, residual, weight, eps):
    """(s, y): s = x + residual, y = s * weight / sqrt(mean(s^2) + eps)."""
    s = sum(np.asarray(a, dtype=np.float64) for a in (x, residual) if a is not None)
    y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return s, y if weight is None else y * np.asarray(weight, dtype=np.float64)


def silu_mul(gate, up):
    gate, up = np.asarray(gate, dtype=np.float64), np.asarray(up, dtype=np.float64)
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate)) * up


def in_codes(y):
    """Rows counted in their 8-bit steps, not rounded: (y * 127 / max|y|, max|y| / 127)."""
    y = np.asarray(y, dtype=np.float64)
    step = np.abs(y).max(-1, keepdims=True) / 127
    return y / np.where(step > 0, step, 1), step[..., 0]


def sums(x, w):
    """Exact integer sums of 8-bit rows x [m][k] with weights w [n][k]."""
    return np.asarray(x, dtype=np.int64) @ np.asarray(w, dtype=np.int64).T


def product(x, x_scales, w, w_scales):
    return sums(x, w) * np.asarray(x_scales, np.float64)[:, None] * np.asarray(w_scales, np.float64)


def route(scores, top_k, normalize):
    """(ids, weights) of rows of scores: the largest first, ties to the lower expert;
    NaN counts as the lowest."""
    ids, weights = [], []
    for z in np.asarray(scores, dtype=np.float64):
        order = sorted(range(len(z)), key=lambda e: (np.isnan(z[e]), 0 if np.isnan(z[e]) else -z[e], e))[:top_k]
        bad = np.isnan(z).any() or z.max() == np.inf or z.max() == -np.inf
        p = np.full(len(z), np.nan) if bad else np.exp(z - z.max())
        total = p[order].sum() if normalize else p.sum()
        ids.append(order)
        weights.append(p[order] / total)
    return np.array(ids, dtype=np.int32), np.array(weights)


def experts(x, x_scales, gate, up, down, ids, weights, near):
    """y of an expert layer, and how far each value may be off because a value of h
    lies within `near` of a step of the border between two codes, which may then be
    either.  gate, up, down: (codes [experts][n][k], scales [experts][n])."""
    m, hidden = len(x), down[0].shape[1]
    y, slack = np.zeros((m, hidden)), np.zeros((m, hidden))
    for i in range(m):
        for e, wt in zip(ids[i], weights[i]):
            if e == -1:
                continue
            if not 0 <= e < len(gate[0]):
                y[i] = np.nan
                continue
            a = product(x[i:i + 1], x_scales[i:i + 1], gate[0][e], gate[1][e])
            b = product(x[i:i + 1], x_scales[i:i + 1], up[0][e], up[1][e])
            h = silu_mul(a, b)[0]
            if not np.isfinite(h).all():
                y[i] = np.nan
                continue
            c, step = in_codes(h)
            d = down[0][e].astype(np.float64) * np.asarray(down[1][e], np.float64)[:, None]
            border = np.abs(np.abs(c - np.trunc(c)) - 0.5) < near
            y[i] += wt * step * (d @ np.rint(c))
            slack[i] += abs(wt) * step * (np.abs(d) @ border)
    return y, slack
