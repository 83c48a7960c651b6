"""Dense product with its epilogue (test infrastructure only), in float64:
out = act(x w^T + bias) + residual and its gradients (include/moe.h,
moe_linear)."""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(act: str, z: np.ndarray) -> np.ndarray:
    if act == "none":
        return z
    if act == "relu":
        return np.maximum(z, 0)
    if act == "silu":
        return z / (1 + np.exp(-z))
    if act == "gelu":
        return z * (1 + _erf(z / math.sqrt(2))) / 2
    if act == "gelu_tanh":
        return z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))) / 2
    raise ValueError(act)


def derivative(act: str, z: np.ndarray) -> np.ndarray:
    if act == "none":
        return np.ones_like(z)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        e = np.exp(-z)
        return (1 + e + z * e) / (1 + e) ** 2
    if act == "gelu":
        return (1 + _erf(z / math.sqrt(2))) / 2 + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return (1 + t) / 2 + z * (1 - t * t) / 2 * c * (1 + 3 * 0.044715 * z ** 2)
    raise ValueError(act)


def product(x, w, bias=None):
    z = x @ w.T
    return z if bias is None else z + bias


def apply(act, z, residual=None):
    n = z.shape[1] // 2
    y = activation("silu", z[:, :n]) * z[:, n:] if act == "swiglu" else activation(act, z)
    return y if residual is None else y + residual


def dz(act, d_out, pre):
    """d loss / d (x w^T + bias)."""
    if act == "swiglu":
        n = d_out.shape[1]
        gate, up = pre[:, :n], pre[:, n:]
        return np.concatenate([d_out * up * derivative("silu", gate), d_out * activation("silu", gate)], axis=1)
    return d_out if act == "none" else d_out * derivative(act, pre)
