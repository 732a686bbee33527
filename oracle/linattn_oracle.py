"""fp64 oracle of linear attention with one decay per head, one token at a time (numpy).

Per batch row b and head h:  S = exp(a_h) S + k_t v_t^T,  y_t = scale q_t^T S.
q [B, L, Hq, dk], k [B, L, Hk, dk], v [B, L, Hv, dv]; H = len(a); head h reads row
h // (H // Hq) of q, and so on.  lengths [B]: tokens of each row; y is 0 behind them.
"""
from __future__ import annotations

import numpy as np


def _heads(t, H):
    return np.repeat(np.asarray(t, np.float64), H // t.shape[2], axis=2)


def _fold(t, heads):
    B, L, H, D = t.shape
    return t.reshape(B, L, heads, H // heads, D).sum(3)


def _setup(q, k, v, a, h0, lengths):
    a = np.asarray(a, np.float64)
    H = a.size
    q, k, v = _heads(q, H), _heads(k, H), _heads(v, H)
    B, L = q.shape[:2]
    S = np.zeros((B, H, q.shape[3], v.shape[3])) if h0 is None else np.array(h0, np.float64)
    n = np.full(B, L) if lengths is None else np.clip(np.asarray(lengths, np.int64), 0, L)
    return q, k, v, np.exp(a)[:, None, None], S, n


def linattn(q, k, v, a, scale, h0=None, lengths=None):
    """y [B, L, H, dv] and the last state [B, H, dk, dv]."""
    q, k, v, lam, S, n = _setup(q, k, v, a, h0, lengths)
    B, L, H = q.shape[:3]
    y = np.zeros((B, L, H, v.shape[3]))
    for t in range(L):
        on = n > t
        S[on] = lam * S[on] + k[on, t, :, :, None] * v[on, t, :, None, :]
        y[on, t] = scale * np.einsum("bhi,bhij->bhj", q[on, t], S[on])
    return y, S


def linattn_bwd(q, k, v, a, scale, h0=None, dy=None, dh_last=None, lengths=None):
    """Gradients of sum(dy * y) + sum(dh_last * h_last), as a dict."""
    heads = q.shape[2], k.shape[2], v.shape[2]
    q, k, v, lam, S, n = _setup(q, k, v, a, h0, lengths)
    dy = np.asarray(dy, np.float64)
    B, L, H = q.shape[:3]
    before = np.zeros((L,) + S.shape)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for t in range(L):
        on = n > t
        before[t] = S
        S[on] = lam * S[on] + k[on, t, :, :, None] * v[on, t, :, None, :]
        dq[on, t] = scale * np.einsum("bhij,bhj->bhi", S[on], dy[on, t])
    G = np.zeros_like(S) if dh_last is None else np.array(dh_last, np.float64)
    da = np.zeros(H)
    for t in reversed(range(L)):
        on = n > t
        G[on] += scale * q[on, t, :, :, None] * dy[on, t, :, None, :]
        dk[on, t] = np.einsum("bhij,bhj->bhi", G[on], v[on, t])
        dv[on, t] = np.einsum("bhij,bhi->bhj", G[on], k[on, t])
        da += (G[on] * lam * before[t][on]).sum((0, 2, 3))
        G[on] = lam * G[on]
    return {"dq": _fold(dq, heads[0]), "dk": _fold(dk, heads[1]), "dv": _fold(dv, heads[2]), "dlog_decay": da, "dh0": G}
