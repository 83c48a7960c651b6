"""Microscaled 4-bit rows (test infrastructure only), in float64: elements and
scales from their definitions, and the product with such weights expert by
expert (include/moe.h, moe_mx_quantize, moe_mx_linear)."""
from __future__ import annotations

import numpy as np

from . import linear as OL

#: what the codes 0 .. 15 stand for
ELEMENTS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def element(y: float) -> int:
    """The code of the element next to y, the even code of two as near."""
    a = min(abs(y), 6.0)
    near = np.abs(ELEMENTS[:8] - a)
    best = np.flatnonzero(near == near.min())
    code = next((c for c in best if c % 2 == 0), best[0])
    return int(code) + (8 if np.signbit(y) else 0)


def quantize(x):
    """(q [M, K / 2], scale [M, K / 32]) of float64 rows, block by block."""
    M, K = x.shape
    q, scale = np.zeros((M, K // 2), np.uint8), np.zeros((M, K // 32), np.uint8)
    for m in range(M):
        for b in range(K // 32):
            v = x[m, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                scale[m, b] = 255
                continue
            top = np.abs(v).max()
            e = -127 if top == 0 else max(-127, int(np.frexp(top)[1]) - 1 - 2)
            codes = [element(t) for t in np.ldexp(v, -e)]
            scale[m, b] = e + 127
            q[m, 16 * b:16 * b + 16] = [codes[2 * i] | codes[2 * i + 1] << 4 for i in range(16)]
    return q, scale


def values(q, scale):
    """What packed rows [..., K / 2] with scales [..., K / 32] stand for."""
    codes = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1, 32)
    s = scale.astype(np.int64)[..., None]
    v = np.where(s == 255, np.nan, np.ldexp(ELEMENTS[codes], np.where(s == 255, 0, s - 127)))
    return v.reshape(*q.shape[:-1], -1)


def linear(x, w, offsets, bias, act, out):
    """out with each expert's rows replaced by act(x w[e]^T + bias[e])."""
    out = out.copy()
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            out[lo:hi] = OL.apply(act, OL.product(x[lo:hi], w[e], None if bias is None else bias[e]))
    return out
