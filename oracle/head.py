"""Oracle of the cross entropy through an output head (NumPy, fp64)."""

import numpy as np


def has_label(labels, V):
    return (labels >= 0) & (labels < V)


def loss_grad(X, W, labels, dloss=None):
    """X [T, H], W [V, H] -> (loss, lse, dX, rest, mag): dX's sum consists of
    terms that add up to mag [T, H] in magnitude; rest = 1 - p of the label, formed
    as the sum of the others."""
    T, V = X.shape[0], W.shape[0]
    l = X @ W.T
    top = l.max(axis=1, keepdims=True)
    p = np.exp(l - top)
    lse = top[:, 0] + np.log(p.sum(axis=1))
    has = has_label(labels, V)
    at = np.where(has, labels, 0)
    rows = np.arange(T)
    mine = p[rows, at]
    others = p.copy()
    others[rows, at] = 0.0
    rest = others.sum(axis=1)
    with np.errstate(divide="ignore"):
        loss = np.where(mine > 1e-200, np.log1p(rest / np.maximum(mine, 1e-200)), lse - l[rows, at])
    loss = np.where(has, loss, 0.0)
    if dloss is None:
        return loss, lse
    total = rest + mine
    rest = rest / total
    g = np.where(has, dloss, 0.0)[:, None]
    others /= total[:, None]
    dX = g * (others @ W - rest[:, None] * W[at])
    mag = np.abs(g) * (others @ np.abs(W) + rest[:, None] * np.abs(W[at]))
    return loss, lse, dX, rest, mag
