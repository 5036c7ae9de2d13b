"""Float64 references of the training-step operators, written from their definitions (NumPy, no code of the library), with
the rounding errors that float32 evaluation may add, followed term by term."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of float32


# ------------------------------------------------------------------ gated linear recurrence
def gate(z, kind):
    """(a, w, da/dz, relative error of a or 1 - a, whichever is smaller, and of w).

    An exponential's argument is rounded twice before the hardware's exp2 (1 ulp), so that it is off by |z| 2U + 2U; the
    sums and quotients behind it add four roundings, the series of 1 - exp(-z) eight."""
    z = z.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "rate":
            a = np.exp(-z)
            w, slope = np.ones_like(z), -a
        else:
            a, w = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
            slope = a * w
        d = np.where(np.isfinite(z), (2 * np.minimum(np.abs(z), 110.0) + 12) * U, 0.0)
    return a, w, slope, d


def scan(z, x, kind, bounds, state_in=None, dh=None, dstate_out=None):
    """Everything that the operator returns and, under the same names with a "~", bounds of the float32 errors."""
    T, C = z.shape
    n = len(bounds) - 1
    a, w, slope, d = gate(z, kind)
    x = x.astype(np.float64)
    f = 0.0 if kind == "rate" else d  # relative error of w
    h, eh, before, ebefore, size = (np.zeros((T, C)) for _ in range(5))
    out = {"state_out": np.zeros((n, C)), "~state_out": np.zeros((n, C)), "dstate_in": np.zeros((n, C)), "~dstate_in": np.zeros((n, C))}
    small = np.minimum(a, np.abs(1 - a))
    for s, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        v = np.zeros(C) if state_in is None else state_in[s].astype(np.float64)
        E, e = np.abs(v), np.zeros(C)
        for t in range(lo, hi):
            before[t], ebefore[t], size[t] = v, e, E
            # the decay's own error, a product and a sum, the input's weight; twice where segments are joined
            e = a[t] * e + 2 * ((small[t] * d[t] + 2 * a[t] * U) * E + (f[t] if np.ndim(f) else f) * np.abs(w[t] * x[t]))
            v = a[t] * v + w[t] * x[t]
            E = a[t] * E + np.abs(w[t] * x[t])
            e = e + 4 * U * E
            h[t], eh[t] = v, e
        out["state_out"][s], out["~state_out"][s] = v, e
    out.update({"h": h, "~h": eh})
    if dh is None:
        return out
    dh = dh.astype(np.float64)
    dz, edz, dx, edx = (np.zeros((T, C)) for _ in range(4))
    for s, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        mu = np.zeros(C) if dstate_out is None else dstate_out[s].astype(np.float64)
        M, e = np.abs(mu), np.zeros(C)
        for t in range(hi - 1, lo - 1, -1):
            lam, L = dh[t] + mu, np.abs(dh[t]) + M
            e = e + 2 * U * L
            dx[t], edx[t] = w[t] * lam, w[t] * e + w[t] * L * (d[t] + 4 * U)
            g = before[t] if kind == "rate" else before[t] - x[t]
            G = size[t] if kind == "rate" else size[t] + np.abs(x[t])
            # a's own relative error is d also where 1 - a is the smaller
            dz[t] = slope[t] * g * lam
            edz[t] = np.abs(slope[t]) * (ebefore[t] * L + G * e + G * L * (2 * d[t] + 8 * U))
            e = a[t] * e + 2 * (small[t] * d[t] + 3 * a[t] * U) * L
            mu, M = a[t] * lam, a[t] * L
        out["dstate_in"][s], out["~dstate_in"][s] = mu, e
    out.update({"dgate": dz, "~dgate": edz, "dx": dx, "~dx": edx})
    return out


# ------------------------------------------------------------------ linear softmax cross entropy
def cross_entropy(x, table, targets, scale, dloss=None, dlse=None, bf16=False):
    """loss, lse, dx, dtable and, with a "~", bounds of the errors of float32 sums (bf16: of factors G rounded to it)."""
    x, table = x.astype(np.float64), table.astype(np.float64)
    T, (V, D) = x.shape[0], table.shape
    inside = (targets >= 0) & (targets < V)
    x = np.where(inside[:, None], x, 0.0)
    y = np.where(inside, targets, 0)
    rows = np.arange(T)
    l = scale * (x @ table.T)
    # a sum of D products of random signs: 8 sqrt(D) roundings of its terms' magnitudes, and the scale's
    el = abs(scale) * (np.abs(x) @ np.abs(table).T) * (8 * np.sqrt(D) + 4) * U
    m = l.max(1, keepdims=True)
    p = np.exp(l - m)
    z = p.sum(1, keepdims=True)
    lse = (m + np.log(z))[:, 0]
    p /= z
    # the logits' errors by weight (at most the largest), exponents rounded at |l - m| 2U + 4U, sums, log, two additions
    ee = 3 * U * np.abs(l - m) + 4 * U
    else_ = (p * (el + ee)).sum(1) * 2 + el.max(1) * 0.5 + (8 * np.sqrt(V) + 8) * U + 4 * U * (np.abs(lse) + np.abs(m[:, 0]))
    loss = lse - l[rows, y]
    out = {"lse": np.where(inside, lse, 0.0), "~lse": np.where(inside, else_, 0.0), "loss": np.where(inside, loss, 0.0),
           "~loss": np.where(inside, else_ + el[rows, y] + 2 * U * (np.abs(lse) + np.abs(l[rows, y])), 0.0)}
    if dloss is None:
        return out
    d = scale * np.where(inside, dloss, 0.0).astype(np.float64)[:, None]
    f = d + (0.0 if dlse is None else scale * np.where(inside, dlse, 0.0).astype(np.float64)[:, None])
    hit = np.zeros((T, V))
    hit[rows, y] = 1.0
    G = f * p - d * hit
    eG = np.abs(f) * p * (el + else_[:, None] + 3 * U * np.abs(l - lse[:, None]) + 8 * U) + 2 * U * np.abs(d) * hit
    eG = eG + np.abs(G) * (2.0 ** -8 if bf16 else 0.0)
    eG = np.where(inside[:, None], eG, 0.0)
    out["dx"], out["dtable"] = G @ table, G.T @ x
    out["~dx"] = eG @ np.abs(table) + (np.abs(G) @ np.abs(table)) * (8 * np.sqrt(V) + 4) * U
    out["~dtable"] = eG.T @ np.abs(x) + (np.abs(G).T @ np.abs(x)) * (8 * np.sqrt(T) + 4) * U
    return out


# ------------------------------------------------------------------ AdamW
def adamw(p, g, m, v, lr, b1, b2, eps, wd, step):
    """New p, m, v in 64 bits, and a bound of p's float32 error."""
    p, g, m, v = (t.astype(np.float64) for t in (p, g, m, v))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    size = b1 * np.abs(m) + (1 - b1) * np.abs(g)
    move = lr / (1 - b1 ** step) / (np.sqrt(v) / np.sqrt(1 - b2 ** step) + eps)
    keep = 1 - lr * wd
    new = keep * p - move * m
    err = 3 * U * np.abs(p) + move * (np.abs(m) * 16 * U + 4 * U * (size + np.abs(g))) + U * np.abs(new)
    return new, m, v, err
