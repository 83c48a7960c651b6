"""Routing (test infrastructure only): the top-k experts and gate weights of
every token from its logits, and the weights' gradient with respect to the
logits, from their definitions in float64 (include/moe.h, moe_route)."""
from __future__ import annotations

import numpy as np


def scores(z: np.ndarray, kind: str) -> np.ndarray:
    """softmax over the experts, or a sigmoid of each; rows of -inf give zeros."""
    z = np.asarray(z, dtype=np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
    out = np.zeros_like(z)
    for t in range(z.shape[0]):
        live = ~np.isneginf(z[t])
        if live.any():
            e = np.exp(z[t, live] - z[t, live].max())
            out[t, live] = e / e.sum()
    return out


def route(z, k, kind="softmax", bias=None, renorm=False, n_group=1, topk_group=0, top2=False, scale=1.0):
    """(ids [T, k] int32, weights [T, k] float64), token by token."""
    z = np.asarray(z, dtype=np.float64)
    T, E = z.shape
    s = scores(z, kind)
    size, keep = E // n_group, topk_group or n_group
    ids = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        c = s[t] + (0 if bias is None else np.asarray(bias, np.float64))
        c = np.where(np.isneginf(z[t]), -np.inf, c)
        if n_group > 1:
            parts = [sorted(c[g * size:(g + 1) * size], reverse=True) for g in range(n_group)]
            value = [(-np.inf if np.isneginf(p[1]) else p[0] + p[1]) if top2 else p[0] for p in parts]
            kept = sorted(range(n_group), key=lambda g: (-value[g], g))[:keep]
            for g in range(n_group):
                if g not in kept:
                    c[g * size:(g + 1) * size] = -np.inf
        order = sorted(range(E), key=lambda e: (-c[e], e))[:k]
        ids[t] = order
        w[t] = [0.0 if np.isneginf(c[e]) else s[t, e] for e in order]
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale


def weights_of(z, ids, held, kind="softmax", renorm=False, scale=1.0):
    """The weights as a function of the logits alone, for fixed ids; `held`
    marks the slots that are not constants at 0."""
    s = scores(z, kind)
    w = np.where(held, np.take_along_axis(s, ids.astype(np.int64), 1), 0.0)
    if renorm:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return w * scale


def route_backward(z, ids, held, g, kind="softmax", renorm=False, scale=1.0):
    """d_logits [T, E]: the weights' Jacobian transposed times g, built slot by
    slot from d s_i / d z_e = s_i ([i = e] - s_e) (softmax) or s_i (1 - s_i) [i = e]."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    s = scores(z, kind)
    out = np.zeros((T, E))
    for t in range(T):
        slots = [j for j in range(ids.shape[1]) if held[t, j]]
        total = sum(s[t, ids[t, j]] for j in slots) if renorm else 1.0
        mean = sum(g[t, j] * s[t, ids[t, j]] for j in slots) / total if renorm and slots else 0.0
        for j in slots:
            i = ids[t, j]
            ds = scale * (g[t, j] - mean) / total      # d loss / d s_i through slot j
            if kind == "sigmoid":
                out[t, i] += ds * s[t, i] * (1 - s[t, i])
            else:
                out[t] -= ds * s[t, i] * s[t]
                out[t, i] += ds * s[t, i]
    return out
