"""Oracle of the 8-bit format and its linear layer (NumPy, fp64).

Format: blocks of 128 x 128 weights (smaller at the edges); scale 2^e, e the
least integer >= -127 with max|w| 2^-e <= 448, byte e + 127 (0 for a block of
zeros); codes are OCP e4m3 of w 2^-e, rounded to nearest even.  Activations:
the same per row and 128 columns.
"""

import numpy as np

BLOCK = 128


def e4m3_values():
    """The value of each of the 256 codes (NaN at 0x7f and 0xff)."""
    c = np.arange(256)
    sign = np.where(c & 0x80, -1.0, 1.0)
    ex, fr = (c >> 3) & 15, (c & 7)
    mag = np.where(ex == 0, fr * 2.0 ** -9, (8 + fr) * np.exp2(ex - 10.0))
    return np.where((c & 0x7f) == 0x7f, np.nan, sign * mag)


def encode(x):
    """fp64 values with |x| <= 448 -> codes, by search: the nearest of the 127
    magnitudes, ties to the even code."""
    mags = e4m3_values()[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(mags, a, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def scale_exponent(amax):
    """The least e >= -127 with amax 2^-e <= 448 (-127 for 0), by counting up."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127, dtype=np.int64)
    while True:
        over = amax > 448.0 * np.exp2(e.astype(np.float64))
        if not over.any():
            return e
        e = e + over


def quantize(w):
    """[R, C] -> (codes uint8 [R, C], scale bytes)."""
    w = np.asarray(w, dtype=np.float64)
    R, C = w.shape
    codes = np.zeros((R, C), dtype=np.uint8)
    scales = np.zeros((-(-R // BLOCK), -(-C // BLOCK)), dtype=np.uint8)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            b = w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            e = int(scale_exponent(np.abs(b).max()))
            scales[i, j] = e + 127
            codes[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = encode(b * 2.0 ** -e)
    return codes, scales


def dequantize(codes, scales):
    """fp64 values code 2^e."""
    v = e4m3_values()[codes]
    f = np.exp2(scales.astype(np.float64) - 127)
    f = np.repeat(np.repeat(f, BLOCK, 0), BLOCK, 1)[:codes.shape[0], :codes.shape[1]]
    return v * f


def quantized_rows(x):
    """x with every row's 128 columns quantized and back (fp64)."""
    x = np.asarray(x, dtype=np.float64)
    out = np.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        b = x[:, c:c + BLOCK]
        f = np.exp2(scale_exponent(np.abs(b).max(axis=1)).astype(np.float64))[:, None]
        out[:, c:c + BLOCK] = e4m3_values()[encode(b / f)] * f
    return out


def linear_fwd(Wh, X, A, B, r, alpha):
    Y = quantized_rows(X) @ Wh.T
    return Y + (alpha / r) * ((X @ A.T) @ B.T) if r else Y


def linear_bwd(Wh, X, dY, A, B, r, alpha):
    dX = quantized_rows(dY) @ Wh
    if not r:
        return dX, None, None
    s, V = alpha / r, dY @ B
    return dX + s * (V @ A), s * (V.T @ X), s * (dY.T @ (X @ A.T))
