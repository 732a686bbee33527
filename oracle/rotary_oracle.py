"""fp64 oracle of rotary positions and head norms (numpy): each pair as a 2x2 matrix, written out per pair.

x [T, heads, dim], positions [T], freqs [pairs] (radians a position).
"""
from __future__ import annotations

import numpy as np


def columns(pairs, interleaved):
    """Columns (a, b) of every pair."""
    j = np.arange(pairs)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)


def turn(x, positions, freqs, interleaved=False, magnitude=1.0, back=False):
    x = np.array(x, np.float64)
    a, b = columns(len(freqs), interleaved)
    th = np.asarray(positions, np.longdouble)[:, None] * np.asarray(freqs, np.longdouble)
    c, s = (f(th).astype(np.float64)[:, None] * magnitude for f in (np.cos, np.sin))
    if back:
        s = -s
    u, v = x[..., a].copy(), x[..., b].copy()
    x[..., a] = u * c - v * s
    x[..., b] = v * c + u * s
    return x


def turn_size(x, freqs, interleaved=False, magnitude=1.0):
    """What every output of a turn is a sum of, in absolute values: |u| + |v| of its pair (an error of an angle
    moves the other column's share in)."""
    x = np.abs(np.array(x, np.float64))
    a, b = columns(len(freqs), interleaved)
    t = magnitude * (x[..., a] + x[..., b])
    x[..., a] = t
    x[..., b] = t
    return x


def norm(x, w=None, eps=1e-6):
    """x / sqrt(mean(x^2) + eps) * w, and the first factor's reciprocal root."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * (1.0 if w is None else np.asarray(w, np.float64)), r


def norm_bwd(x, w, g, eps=1e-6):
    """Gradients (dx, dw) of sum(g * norm(x))."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    e = g * (1.0 if w is None else np.asarray(w, np.float64))
    dx = r * e - x * r ** 3 * (e * x).mean(-1, keepdims=True)
    return dx, (g * x * r).reshape(-1, x.shape[-1]).sum(0)
