"""fp64 oracle of the operators between features and Gaussian parameters: linear,
gated and rms_norm with their gradients, in plain numpy (tests only).

    linear    y = act(x W^T + b) + r
    gated     h = act(x Wg^T) * (x Wu^T)
    rms_norm  s = x + r,  y = s / sqrt(mean s^2 + eps) * w
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])
E4M3_MAX, MIN_SCALE = 448.0, 2.0 ** -126


def act(z, kind):
    """(value, derivative) of an activation."""
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "none":
            return z, np.ones_like(z)
        if kind == "relu":
            return np.where(z < 0, 0.0, z), (z > 0).astype(np.float64)
        if kind == "silu":
            t = 1 / (1 + np.exp(-z))
            return z * t, t + z * t * (1 - t)
        if kind == "gelu":
            p = 0.5 * (1 + _erf(z / math.sqrt(2.0)))
            return z * p, p + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if kind == "gelu_tanh":
            c = math.sqrt(2 / math.pi)
            t = np.tanh(c * (z + 0.044715 * z ** 3))
            return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    raise ValueError(kind)


def linear(x, w, b=None, r=None, kind="none"):
    z = x @ w.T + (0 if b is None else b)
    return act(z, kind)[0] + (0 if r is None else r)


def linear_bwd(dy, x, w, b=None, kind="none"):
    """(dx, dw, db)."""
    z = x @ w.T + (0 if b is None else b)
    dz = dy * act(z, kind)[1]
    return dz @ w, dz.T @ x, dz.sum(0)


def gated(x, wg, wu, kind="silu"):
    return act(x @ wg.T, kind)[0] * (x @ wu.T)


def gated_bwd(dh, x, wg, wu, kind="silu"):
    """(dx, dwg, dwu)."""
    g, u = x @ wg.T, x @ wu.T
    a, s = act(g, kind)
    dg, du = dh * u * s, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x


def rms_norm(x, w, r=None, eps=1e-6):
    """(y, s)."""
    s = x if r is None else x + r
    return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * w, s


def rms_norm_bwd(dy, s, w, ds=None, eps=1e-6):
    """(dx, dw); dx is the residual's gradient too."""
    m = np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    p = dy * w
    dx = p / m - s * (p * s).mean(-1, keepdims=True) / m ** 3
    return dx if ds is None else dx + ds, (dy * s / m).sum(0)


def row_scales(y):
    """The scale of each row in 8 bits."""
    return np.maximum(np.abs(y).max(-1) / E4M3_MAX, MIN_SCALE)
