"""Oracle of the mixture-of-experts operators (NumPy, fp64)."""

import numpy as np


def route(logits, k, renormalize):
    """ids (largest first, ties to the lower index, NaN above every number) and
    weights of each row."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    ids = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted(range(E), key=lambda e: (0, 0.0, e) if np.isnan(l[t, e]) else (1, -l[t, e], e))
        ids[t] = order[:k]
        row = l[t]
        if np.all(row == -np.inf):
            continue
        with np.errstate(invalid="ignore"):
            x = np.exp(row - row[ids[t, 0]])
            w[t] = x[ids[t]] / (x[ids[t]].sum() if renormalize else x.sum())
    return ids, w


def route_bwd(logits, ids, dw, renormalize):
    l = np.asarray(logits, dtype=np.float64)
    out = np.zeros_like(l)
    for t in range(l.shape[0]):
        row = l[t].copy()
        if renormalize:
            keep = np.zeros(l.shape[1], dtype=bool)
            keep[ids[t]] = True
            row[~keep] = -np.inf
        if np.all(row == -np.inf):
            continue
        p = np.exp(row - row.max())
        p /= p.sum()
        g = np.zeros(l.shape[1])
        g[ids[t]] = dw[t]
        out[t] = p * (g - (g * p).sum())
    return out


def experts(gate_up, down, X, ids, weights):
    """gate_up [E, 2, I, H], down [E, H, I], fp64; (Y, sums of magnitudes of the
    down products, for error bounds)."""
    E = gate_up.shape[0]
    Y = np.zeros_like(X)
    mag = np.zeros_like(X)
    for t in range(X.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            g, u = gate_up[e, 0] @ X[t], gate_up[e, 1] @ X[t]
            h = g / (1 + np.exp(-g)) * u
            Y[t] += weights[t, j] * (down[e] @ h)
            mag[t] += abs(weights[t, j]) * (np.abs(down[e]) @ np.abs(h))
    return Y, mag
