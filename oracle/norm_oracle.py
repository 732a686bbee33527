"""fp64 oracle of the group norm, channels last (numpy).

x [N, L, C], groups of C / G consecutive channels; mean and variance over a group's L * C / G
values:  u = (x - mean) / sqrt(var + eps) * w + b,  y = act(u) * silu(z).
"""
from __future__ import annotations

import numpy as np


def sigmoid(t):
    return 0.5 * (1.0 + np.tanh(0.5 * t))


def parts(x, groups, w=None, b=None, z=None, eps=1e-5, silu=False):
    """xh, rstd, u, act(u), gate: what forward and backward are made of ([N, L, C]; rstd [N, 1, G, 1])."""
    x = np.asarray(x, np.float64)
    N, L, C = x.shape
    t = x.reshape(N, L, groups, C // groups)
    t = t - t.mean((1, 3), keepdims=True)
    rstd = 1.0 / np.sqrt((t * t).mean((1, 3), keepdims=True) + eps)
    xh = (t * rstd).reshape(N, L, C)
    u = xh * (1.0 if w is None else np.asarray(w, np.float64)) + (0.0 if b is None else np.asarray(b, np.float64))
    a = u * sigmoid(u) if silu else u
    gate = 1.0 if z is None else np.asarray(z, np.float64) * sigmoid(np.asarray(z, np.float64))
    return xh, rstd, u, a, gate


def groupnorm(x, groups, w=None, b=None, z=None, eps=1e-5, silu=False):
    _, _, _, a, gate = parts(x, groups, w, b, z, eps, silu)
    return a * gate


def groupnorm_bwd(x, groups, w=None, b=None, z=None, dy=None, eps=1e-5, silu=False):
    """Gradients of sum(dy * y): dx, dw, dbias, dz."""
    xh, rstd, u, a, gate = parts(x, groups, w, b, z, eps, silu)
    dy = np.asarray(dy, np.float64)
    N, L, C = xh.shape
    g = dy * gate
    if silu:
        s = sigmoid(u)
        g = g * s * (1.0 + u * (1.0 - s))
    e = (g * (1.0 if w is None else np.asarray(w, np.float64))).reshape(N, L, groups, C // groups)
    n = xh.reshape(e.shape)
    dx = rstd * (e - e.mean((1, 3), keepdims=True) - n * (e * n).mean((1, 3), keepdims=True))
    out = {"dx": dx.reshape(xh.shape), "dw": (g * xh).sum((0, 1)), "dbias": g.sum((0, 1)), "dz": None}
    if z is not None:
        z = np.asarray(z, np.float64)
        s = sigmoid(z)
        out["dz"] = dy * a * s * (1.0 + z * (1.0 - s))
    return out
