"""fp64 oracle of a Mamba-2 layer's served mixer (numpy): convolution, SiLU and multi-head scan, one token of one
sequence after another.  Beside every value it carries a bound: the same formulas over absolute values, with half the
decays' exponents (see `hats`).
"""
from __future__ import annotations

import numpy as np


def sigmoid(t):
    return 0.5 * (1.0 + np.tanh(0.5 * t))


def softplus(t):
    return np.logaddexp(0.0, t)


def mixer(c, ends=None):
    """c: dict with xbc [T, C], delta [T, H], z [T, H, P] or None, A, D, delta_bias [H] (the last two or None), w [C, W], bias [C]
    or None, h [slots, H, P, N], conv_state [slots, C, W - 1], offsets [S + 1], slots [S], fresh [S], G, softplus; all in
    64 bits.  Returns y [T, H, P] (NaN in rows of no sequence), h and conv_state afterwards, and the bounds of y and h.

    hats: with x^ = |x| + 1.1 (sum |w xbc| + |bias|) (what rounding the convolution's sum can move silu by) and so on,
    S^ = sqrt(decay) S^ + dt x^ B^ and y^ = (S^ C^ + |D| x^) |silu z|: an error of a decay's exponent X, relative to X,
    moves exp(-X) by X exp(-X) <= 1.3 exp(-X / 2) of it.
    """
    f = lambda n: None if c[n] is None else np.asarray(c[n], np.float64)  # noqa: E731
    xbc, delta, z, A, w = f("xbc"), f("delta"), f("z"), f("A"), f("w")
    h, st = f("h").copy(), f("conv_state").copy()
    hh = np.abs(h)
    (T, C), (H, P, N), W, G = xbc.shape, h.shape[1:], w.shape[1], c["G"]
    D = np.zeros(H) if c["D"] is None else f("D")
    bias = np.zeros(C) if c["bias"] is None else f("bias")
    dbias = np.zeros(H) if c["delta_bias"] is None else f("delta_bias")
    y, yh = np.full((T, H, P), np.nan), np.zeros((T, H, P))
    rep = np.arange(H) // (H // G)
    for s in range(len(c["slots"])):
        slot, a, b = int(c["slots"][s]), int(c["offsets"][s]), int(c["offsets"][s + 1])
        kept = 0 <= slot < h.shape[0]
        old = kept and not c["fresh"][s]
        S = h[slot].copy() if old else np.zeros((H, P, N))
        Sh = np.abs(S)
        win = st[slot].copy() if old else np.zeros((C, W - 1))
        for t in range(a, b):
            win = np.concatenate([win, xbc[t][:, None]], 1)
            v = (win * w).sum(1) + bias
            vh = (np.abs(win * w)).sum(1) + np.abs(bias)
            v, vh = v * sigmoid(v), np.abs(v * sigmoid(v)) + 1.1 * vh
            win = win[:, 1:]
            cut = lambda m: (m[:H * P].reshape(H, P), m[H * P:H * P + G * N].reshape(G, N)[rep], m[H * P + G * N:].reshape(G, N)[rep])  # noqa: E731
            (x, B, Cv), (xh, Bh, Ch) = cut(v), cut(vh)
            dt = delta[t] + dbias
            dt = softplus(dt) if c["softplus"] else dt
            dec = np.exp(dt * A)[:, None, None]
            S = dec * S + (dt[:, None] * x)[:, :, None] * B[:, None]
            Sh = np.sqrt(dec) * Sh + (np.abs(dt)[:, None] * xh)[:, :, None] * Bh[:, None]
            g = np.ones((H, P)) if z is None else z[t] * sigmoid(z[t])
            y[t] = ((S * Cv[:, None]).sum(-1) + D[:, None] * x) * g
            yh[t] = ((Sh * Ch[:, None]).sum(-1) + np.abs(D)[:, None] * xh) * np.abs(g)
        if kept:
            h[slot], hh[slot], st[slot] = S, Sh, win
    return {"y": y, "h": h, "conv_state": st, "y_hat": yh, "h_hat": hh}
