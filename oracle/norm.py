"""Oracle of the root-mean-square norm (NumPy, fp64)."""

import numpy as np


def fwd(h, w, eps):
    """(y, rstd) of rows h."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def bwd(dy, h, w, rstd, dres=None):
    """(dh, dw), and the magnitudes that their sums consist of."""
    n, g = h * rstd[:, None], dy * w
    r = rstd[:, None]
    dh = r * (g - n * (g * n).mean(axis=1, keepdims=True))
    mag = r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    if dres is not None:
        dh, mag = dh + dres, mag + np.abs(dres)
    return dh, (dy * n).sum(axis=0), mag, np.abs(dy * n).sum(axis=0)
