"""Float64 references of the sequence layers, written from their definitions
(NumPy, no code of the library): decayed attention token by token and pair by
pair, layer norm, embedding."""
from __future__ import annotations

import numpy as np


def weight(rate: float, lag):
    """exp(-rate lag), 1 at lag 0 whatever the rate."""
    lag = np.asarray(lag, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        return np.where(lag == 0, 1.0, np.exp(-rate * lag))


def attn_scan(q, k, v, rate, bounds, scale, state_in=None):
    """o (T, H, dv) and the final states (N, H, dk, dv), one token after the other."""
    T, H, dk = q.shape
    g, dv = H // k.shape[1], v.shape[2]
    q, k, v = (x.astype(np.float64) for x in (q, np.repeat(k, g, 1), np.repeat(v, g, 1)))
    o = np.zeros((T, H, dv))
    final = np.zeros((len(bounds) - 1, H, dk, dv))
    w = weight_per_head(rate, 1)
    for s, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        S = np.zeros((H, dk, dv)) if state_in is None else state_in[s].astype(np.float64)
        for t in range(a, b):
            S = w[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
        final[s] = S
    return o, final


def weight_per_head(rate, lag):
    return np.array([weight(float(r), lag) for r in rate])


def attn_pairs(q, k, v, rate, go, bounds, scale, state_in=None, dstate_out=None, absolute=False):
    """Every gradient from sums over pairs (i, j); with absolute=True the same sums of the terms'
    magnitudes, the size that rounding errors are measured against.  Also the forward output."""
    T, H, dk = q.shape
    kv, dv = k.shape[1], v.shape[2]
    g = H // kv
    f = np.abs if absolute else (lambda x: x)
    q, k, v, go = (f(x.astype(np.float64)) for x in (q, np.repeat(k, g, 1), np.repeat(v, g, 1), go))
    out = {"o": np.zeros((T, H, dv)), "dq": np.zeros((T, H, dk)), "dk": np.zeros((T, H, dk)), "dv": np.zeros((T, H, dv)),
           "drate": np.zeros(H), "dstate_in": np.zeros((len(bounds) - 1, H, dk, dv)),
           "state_out": np.zeros((len(bounds) - 1, H, dk, dv))}
    sign = 1.0 if absolute else -1.0
    for s, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        L = b - a
        i = np.arange(L)
        lag = i[:, None] - i[None, :]
        for h in range(H):
            r = float(rate[h])
            W = np.where(lag >= 0, weight(r, np.maximum(lag, 0)), 0.0) * scale
            Q, K, V, G = q[a:b, h], k[a:b, h], v[a:b, h], go[a:b, h]
            S0 = np.zeros((dk, dv)) if state_in is None else f(state_in[s, h].astype(np.float64))
            GF = np.zeros((dk, dv)) if dstate_out is None else f(dstate_out[s, h].astype(np.float64))
            P, D = Q @ K.T, G @ V.T
            up, down, whole = weight(r, i + 1) * scale, weight(r, L - 1 - i), weight(r, L)
            out["o"][a:b, h] = (W * P) @ V + up[:, None] * (Q @ S0)
            out["state_out"][s, h] = whole * S0 + (down[:, None] * K).T @ V
            out["dq"][a:b, h] = (W * D) @ K + up[:, None] * (G @ S0.T)
            out["dk"][a:b, h] = (W * D).T @ Q + down[:, None] * (V @ GF.T)
            out["dv"][a:b, h] = (W * P).T @ G + down[:, None] * (K @ GF)
            out["dstate_in"][s, h] = whole * GF + (up[:, None] * Q).T @ G
            out["drate"][h] += sign * ((np.maximum(lag, 0) * W * P * D).sum() + ((i + 1) * up * ((Q @ S0) * G).sum(1)).sum()
                                       + ((L - 1 - i) * down * ((K @ GF) * V).sum(1)).sum() + L * whole * (S0 * GF).sum())
    out["dk"] = out["dk"].reshape(T, kv, g, dk).sum(2)
    out["dv"] = out["dv"].reshape(T, kv, g, dv).sum(2)
    return out


def layer_norm(x, w, b, eps):
    x = x.astype(np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(-1) + eps)
    z = (x - mean[:, None]) * rstd[:, None]
    return z * (1.0 if w is None else w.astype(np.float64)) + (0.0 if b is None else b.astype(np.float64)), mean, rstd


def layer_norm_backward(x, dy, w, eps):
    _, mean, rstd = layer_norm(x, None, None, eps)
    g = dy.astype(np.float64)
    z = (x.astype(np.float64) - mean[:, None]) * rstd[:, None]
    u = g * (1.0 if w is None else w.astype(np.float64))
    dx = rstd[:, None] * (u - u.mean(-1, keepdims=True) - z * (u * z).mean(-1, keepdims=True))
    return dx, (g * z).sum(0), g.sum(0), z


def embedding_backward(ids, dy, vocab, scale):
    out = np.zeros((vocab, dy.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < vocab:
            out[i] += scale * dy[t].astype(np.float64)
    return out
