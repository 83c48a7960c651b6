"""Rows sorted by expert (test infrastructure only): the sort, the copy of
tokens to rows and the weighted sum back with their gradients, slot by slot in
float64 (include/moe.h, moe_sort, moe_permute, moe_unpermute)."""
from __future__ import annotations

import numpy as np


def sort(ids, experts, first=0):
    """(pos [T, k], src [R], offsets [E + 1]), expert by expert."""
    T, k = ids.shape
    pos, src, offsets = np.full((T, k), -1, np.int32), [], [0]
    for e in range(experts):
        for slot in np.flatnonzero(ids.reshape(-1).astype(np.int64) - first == e):
            pos[slot // k, slot % k] = len(src)
            src.append(slot)
        offsets.append(len(src))
    return pos, np.array(src, np.int32), np.array(offsets, np.int32)


def _slots(pos, rows):
    return [(t, j, pos[t, j]) for t in range(pos.shape[0]) for j in range(pos.shape[1]) if 0 <= pos[t, j] < rows]


def permute(x, pos, rows):
    """Rows [R, d] with the tokens' in their places; the others stay."""
    out = rows.copy()
    for t, _, p in _slots(pos, rows.shape[0]):
        out[p] = x[t]
    return out


def unpermute(rows, pos, w=None):
    """(sum, sum of magnitudes) per token."""
    out = np.zeros((pos.shape[0], rows.shape[1]))
    size = np.zeros_like(out)
    for t, j, p in _slots(pos, rows.shape[0]):
        part = rows[p] if w is None else w[t, j] * rows[p]
        out[t] += part
        size[t] += np.abs(part)
    return out, size


def unpermute_backward(rows, pos, w, g, d_rows):
    """(d_rows over the given ones, d_w, magnitudes of d_w's sums)."""
    d_rows, d_w = d_rows.copy(), np.zeros(pos.shape)
    size = np.zeros(pos.shape)
    for t, j, p in _slots(pos, rows.shape[0]):
        d_rows[p] = g[t] if w is None else w[t, j] * g[t]
        d_w[t, j] = (g[t] * rows[p]).sum()
        size[t, j] = np.abs(g[t] * rows[p]).sum()
    return d_rows, d_w, size
