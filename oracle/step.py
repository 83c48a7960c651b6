"""The training step around the sorted rows (test infrastructure only), in
float64: out[t] = sum_j w[t][j] down[e] swiglu(up[e] x[t]), e the expert of slot
(t, j), w the chosen experts' renormalised softmax of the logits, and the gradients
of <g, out>, each from its formula (include/moe.h, moe_route, moe_permute,
moe_linear, moe_unpermute and their gradients).  The rank hosts experts
first .. first + E - 1; slots of others add nothing."""
from __future__ import annotations

import numpy as np

from . import linear as OL
from . import route as OR


def loss(x, up, down, logits, ids, g, first):
    """<g, out>, slot by slot."""
    w = OR.weights_of(logits, ids, np.ones(ids.shape, bool), "softmax", True)
    total = 0.0
    for t, j in np.ndindex(*ids.shape):
        e = ids[t, j] - first
        if 0 <= e < len(up):
            total += w[t, j] * g[t] @ (down[e] @ OL.apply("swiglu", (up[e] @ x[t])[None])[0])
    return total


def gradients(x, up, down, logits, ids, g, first):
    """{"dx", "d_up", "d_down", "d_logits"} of the loss."""
    w = OR.weights_of(logits, ids, np.ones(ids.shape, bool), "softmax", True)
    d = {"dx": np.zeros_like(x), "d_up": np.zeros_like(up), "d_down": np.zeros_like(down)}
    d_w = np.zeros(ids.shape)
    for t, j in np.ndindex(*ids.shape):
        e = ids[t, j] - first
        if not 0 <= e < len(up):
            continue
        z = (up[e] @ x[t])[None]
        h = OL.apply("swiglu", z)[0]
        d_w[t, j] = g[t] @ (down[e] @ h)
        d_y = w[t, j] * g[t]
        d["d_down"][e] += np.outer(d_y, h)
        d_z = OL.dz("swiglu", (down[e].T @ d_y)[None], z)[0]
        d["d_up"][e] += np.outer(d_z, x[t])
        d["dx"][t] += up[e].T @ d_z
    d["d_logits"] = OR.route_backward(logits, ids, np.ones(ids.shape, bool), d_w, "softmax", True)
    return d
