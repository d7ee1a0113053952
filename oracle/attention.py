"""Plain fp64 reference of the attention side of a round: per-head norm and
rotation, 8-bit cache rows, attention over cached and own positions, and the
bookkeeping of a drafted tree.  Written from the definitions, one request and
one head at a time; shares nothing with the HIP path."""
from __future__ import annotations

import numpy as np


def norm_rotate(x, weight, eps, inv_freq, positions, interleaved=False):
    """x [rows][heads][d] -> fp64: x * weight / sqrt(mean(x^2) + eps), then pairs
    of the first 2 * len(inv_freq) dimensions turned by position * inv_freq."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    if inv_freq is None:
        return x
    h = len(inv_freq)
    ang = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s, y = np.cos(ang), np.sin(ang), x.copy()
    first, second = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


def quantise_rows(x):
    """fp32 rows [...][d] -> (int codes, fp32 scale): scale = max|x| / 127, code =
    x * (127 / max|x|) rounded half to even, each step in fp32 as the rule is."""
    x = np.asarray(x, dtype=np.float32)
    top = np.abs(x).max(-1)
    with np.errstate(all="ignore"):
        inv = np.float32(127) / top
        code = np.rint(x * inv[..., None])
        scale = top / np.float32(127)
    bad, tiny = ~np.isfinite(top), ~np.isfinite(inv)
    code = np.where((bad | tiny)[..., None], 0, code).astype(np.int32)
    return code, np.where(bad, np.nan, np.where(tiny, 0, scale)).astype(np.float32)


def attention(q, k, v, cached, masks, scale):
    """q [rows][q_heads][d], k/v [cached + rows][kv_heads][d], masks [rows] ints
    (bit j: sees own row j).  Returns (out [rows][q_heads][d], sum p|v|)."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    rows, hq, d = q.shape
    rep = hq // k.shape[1]
    out, mag = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    for i in range(rows):
        seen = list(range(cached)) + [cached + j for j in range(rows) if masks[i] >> j & 1]
        if not seen:
            continue
        for h in range(hq):
            z = k[seen, h // rep] @ q[i, h] * scale
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h] = p @ v[seen, h // rep]
            mag[i, h] = p @ np.abs(v[seen, h // rep])
    return out, mag


def tree_layout(parents, cache_len):
    """(masks, positions) of one request's nodes; parents of nodes 1 .., -1: not
    there.  A parent that is not below its node makes every mask 0."""
    m = len(parents) + 1
    if any(p < -1 or p > j for j, p in enumerate(parents)):
        return [0] * m, [cache_len] * m
    masks, pos = [1], [cache_len]
    for j, p in enumerate(parents, 1):
        there = p >= 0 and masks[p] != 0
        masks.append(masks[p] | 1 << j if there else 0)
        pos.append(pos[p] + 1 if there else cache_len)
    return masks, pos


def accept_tree_greedy(target, draft, parents):
    """(accept_len, committed, path) of one request, unpadded; (-1, [], []) on a fault."""
    if any(p < -1 or p > j for j, p in enumerate(parents)):
        return -1, [], []
    path = [0]
    while True:
        kids = [j for j, p in enumerate(parents, 1) if p == path[-1] and draft[j - 1] == target[path[-1]]]
        if not kids:
            return len(path), [target[j] for j in path], path
        path.append(kids[0])
