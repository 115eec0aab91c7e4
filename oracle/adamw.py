"""Oracle of the AdamW step with states in 32 or 8 bits (NumPy, fp64)."""

import numpy as np

from . import fp8

BLOCK = 128


def step(p, g, m, v, t, lr, b1, b2, eps, wd):
    """(p, m, v) after step t, all fp64."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    hat_m, hat_v = m / (1 - b1 ** t), v / (1 - b2 ** t)
    return p - lr * wd * p - lr * hat_m / (np.sqrt(hat_v) + eps), m, v


def mix32(x):
    """Two rounds of shift and odd factor, which spread every bit over a word, on uint32 arrays
    (the constants: Austin Appleby's published 32-bit ones, public domain)."""
    x = np.asarray(x, dtype=np.uint32)
    x = (x ^ (x >> np.uint32(16))) * np.uint32(0x85EBCA6B)
    x = (x ^ (x >> np.uint32(13))) * np.uint32(0xC2B2AE35)
    return x ^ (x >> np.uint32(16))


def noise(n, seed, first=0):
    """(u of m, u of sqrt v) for state elements first .. first + n - 1: bytes of the
    hash of the element's pair; first even."""
    i = np.arange(first, first + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        h = mix32((i // 2).astype(np.uint32) ^ mix32(np.array([seed], dtype=np.uint32)))
    odd = (i % 2).astype(np.uint32)
    byte = [(h >> (np.uint32(16) * odd + np.uint32(8 * k))) & np.uint32(255) for k in (0, 1)]
    return [(b.astype(np.float64) + 0.5) / 256 for b in byte]


def distance(y):
    """The distance of e4m3 values at |y|."""
    y = np.abs(np.asarray(y, dtype=np.float64))
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where(y > 0, y, 1.0)))
    return np.where(y < 2.0 ** -6, 2.0 ** -9, np.exp2(np.maximum(e, -6) - 3))


def to8(x, u, keep):
    """State values of one tensor (fp64, padded here to whole blocks) -> (values of
    the codes before scaling, scale bytes, steps): |value| = floor(|y| / step + u)
    step of y = x 2^-e; keep: what is not 0 stays so."""
    n = len(x)
    pad = np.zeros(-(-n // BLOCK) * BLOCK)
    pad[:n] = x
    b = pad.reshape(-1, BLOCK)
    e = fp8.scale_exponent(np.abs(b).max(axis=1))
    y = (b / np.exp2(e.astype(np.float64))[:, None]).reshape(-1)[:n]
    d = distance(y)
    k = np.floor(np.abs(y) / d + u[:n])
    if keep:
        k = np.where(y != 0, np.maximum(k, 1), k)
    return np.sign(y) * k * d, (e + 127).astype(np.uint8), y, d


def from8(codes, scales):
    """Values of codes with one scale byte per block."""
    f = np.repeat(np.exp2(scales.astype(np.float64) - 127), BLOCK)[:len(codes)]
    return fp8.e4m3_values()[codes] * f
