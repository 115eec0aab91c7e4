"""The norm on the GPU at the ends of its range, against oracle/norm.py in 64 bits.

y is one value of fp32 accuracy, rounded once: rstd is within 2^-40 before it is
split in two, the products' remainders are kept, and the last multiply-add rounds at
2^-24.  So y is the bf16 rounding of a value within 2^-23 of the exact one, and rstd, rounded
once, within 2^-24 (1 + 2^-15).  Below fp32's normal range (2^-126) half of its
smallest step, 2^-150, comes in the place of the relative error."""

import numpy as np
import pytest
import torch

import synth
from oracle import nf4 as onf4
from oracle import norm as onorm

from gpu_util import banner, dev_bf16, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu

# each number of lanes a row and chunks a lane
WIDTHS = [64, 192, 512, 1024, 2048, 4096, 8192, 16384]


def _wide(t):
    return onf4.bf16_bits_to_f32(host_bits(t)).astype(np.float64)


def _bits16(x):
    return synth.bf16_bits(x.astype(np.float32))


def _check(h, w, y, rstd, eps):
    ry, rr = onorm.fwd(_wide(h), host(w).astype(np.float64), float(np.float32(eps)))
    assert (np.abs(host(rstd) - rr) <= 2.0 ** -24 * (1 + 2.0 ** -15) * rr + 2.0 ** -150).all()
    # (y in steps of bf16's largest finite value: none of these reaches it)
    lo, hi = (onf4.bf16_bits_to_f32(_bits16(ry * (1 + s * 2.0 ** -23 * np.sign(ry)))) for s in (-1, 1))
    got = _wide(y)
    assert ((got >= lo) & (got <= hi)).all(), np.argwhere((got < lo) | (got > hi))[:5]


@pytest.mark.parametrize("H", WIDTHS)
def test_rows_of_any_finite_size(H):
    """Rows around 2^k up to bf16's largest, whose square sums no fp32 value holds, and
    small ones without eps, whose squares fp32 loses."""
    q = require_gpu()
    banner(f"norm range H={H}")
    w = dev_f32(1 + 0.3 * synth.normal_f32(1, (H,), 1.0))
    base = np.clip(synth.normal_f32(2, (1, H), 1.0), -3.9, 3.9)
    for eps, powers in ((1e-6, (-90, -20, 0, 40, 56, 57, 58, 59, 60, 63, 64, 90, 110, 125)),
                        (0.0, (-120, -100, -74, -63, -60, -20, 0, 59, 64, 125))):
        x = dev_bf16(_bits16(base * np.exp2(np.array(powers, dtype=np.float32))[:, None]))
        y, _, _, rstd = q.qlora_rmsnorm_fwd(x, w, eps=eps)
        _check(x, w, y, rstd, eps)
        zero = torch.zeros_like(x)
        y2, _, h, r2 = q.qlora_rmsnorm_fwd(x, w, residual=zero, eps=eps)
        assert torch.equal(h, x) and torch.equal(y2, y) and torch.equal(r2, rstd)


def test_one_large_value_in_a_row():
    """A row's only value that counts, at each place in turn; the others vanish
    beside it.  |y| there is sqrt(H) w."""
    q = require_gpu()
    banner("norm one large value")
    H = 192
    x = np.full((H, H), 2.0 ** -20, dtype=np.float32)
    x[np.arange(H), np.arange(H)] = -2.0 ** 127
    w = dev_f32(1 + 0.3 * synth.normal_f32(3, (H,), 1.0))
    x = dev_bf16(_bits16(x))
    y, _, _, rstd = q.qlora_rmsnorm_fwd(x, w, eps=1e-6)
    _check(x, w, y, rstd, 1e-6)


@pytest.mark.parametrize("T,H", [(2000, 192), (900, 2048), (512, 8192)])
def test_y_is_rounded_once(T, H):
    """Ordinary rows: no y is further from the exact value's rounding than 2^-23
    of the value explains."""
    q = require_gpu()
    banner(f"norm rounded once {T}x{H}")
    x = synth.normal_f32(T, (T, H), 1.0) * np.exp(synth.normal_f32(T + 1, (T, 1), 1.0))
    w = dev_f32(1 + 0.1 * synth.normal_f32(4, (H,), 1.0))
    x = dev_bf16(_bits16(x))
    y, _, _, rstd = q.qlora_rmsnorm_fwd(x, w, eps=1e-6)
    _check(x, w, y, rstd, 1e-6)


@pytest.mark.parametrize("H", WIDTHS)
def test_gradient_of_large_and_small_rows(H):
    """dh and dw from h and rstd whose product is ordinary, however large h is.  A row's
    sum: 49 roundings of its magnitudes and six more behind it; dw: T + 34 (as
    test_gpu_norm.py).  A subnormal rstd (from 2^126 on) is exact in what is given
    to the oracle."""
    q = require_gpu()
    banner(f"norm gradient range H={H}")
    powers = np.array([-100, -60, 0, 59, 64, 100, 125], dtype=np.float32)
    T = len(powers)
    h = dev_bf16(_bits16(np.clip(synth.normal_f32(5, (T, H), 1.0), -3.9, 3.9) * np.exp2(powers)[:, None]))
    w = dev_f32(1 + 0.3 * synth.normal_f32(6, (H,), 1.0))
    _, _, _, rstd = q.qlora_rmsnorm_fwd(h, w, eps=0.0)
    dy = dev_bf16(_bits16(synth.normal_f32(7, (T, H), 1.0)))
    dh, dw = q.qlora_rmsnorm_bwd(dy, h, w, rstd)
    rdh, rdw, mag, magw = onorm.bwd(_wide(dy), _wide(h), host(w).astype(np.float64), host(rstd).astype(np.float64))
    u = 2.0 ** -24
    # (a dh below bf16's normal range: half of its smallest step, 2^-134)
    assert (np.abs(_wide(dh) - rdh) <= 2.0 ** -8 * np.abs(rdh) + 64 * u * mag + 2.0 ** -133).all()
    assert (np.abs(host(dw) - rdw) <= (T + 34) * u * magw + 1e-38).all()


@pytest.mark.parametrize("H", [64, 576, 4096, 8256])
def test_weights_that_are_not_finite(H):
    """An infinite weight gives an infinite y of the product's sign, a NaN weight NaN, in its
    column alone; 0 times infinity is NaN."""
    q = require_gpu()
    banner(f"norm infinite weight H={H}")
    T, inf = 40, float("inf")
    x = dev_bf16(_bits16(synth.normal_f32(8, (T, H), 1.0)))
    x[3, 1] = 0
    w = dev_f32(1 + 0.3 * synth.normal_f32(9, (H,), 1.0))
    bad = w.clone()
    bad[1], bad[H // 2], bad[H - 1] = inf, -inf, float("nan")
    y, rows, _, rstd = q.qlora_rmsnorm_fwd(x, w, rows8=True)
    yb, _, _, sb = q.qlora_rmsnorm_fwd(x, bad, rows8=True)
    assert torch.equal(sb, rstd)
    keep = torch.ones(H, dtype=torch.bool, device="cuda")
    keep[[1, H // 2, H - 1]] = False
    assert torch.equal(yb[:, keep], y[:, keep])
    s = torch.sign(x.float())
    assert bool(torch.isnan(yb[3, 1])) and bool(torch.isnan(yb[:, H - 1]).all())
    rest = torch.arange(T, device="cuda") != 3
    assert torch.equal(yb[rest, 1].float(), s[rest, 1] * inf) and torch.equal(yb[:, H // 2].float(), s[:, H // 2] * -inf)
    # rows of +-1 without eps: rstd is 1, and no product has a remainder
    ones = torch.where(x >= 0, 1.0, -1.0).to(torch.bfloat16)
    y1, _, _, r1 = q.qlora_rmsnorm_fwd(ones, bad, eps=0.0)
    assert bool((r1 == 1).all()) and torch.equal(y1[:, 1], ones[:, 1] * inf) and torch.equal(y1[:, H // 2], ones[:, H // 2] * -inf)
    # the largest finite weights: y as the formula rounds it, an infinity past bf16's largest
    big = torch.full_like(w, 2.0 ** 127)
    yl = q.qlora_rmsnorm_fwd(x, big)[0]
    ry, _ = onorm.fwd(_wide(x), host(big).astype(np.float64), float(np.float32(1e-6)))
    inside = np.abs(ry) < 2.0 ** 127 * 1.98
    assert (np.abs(_wide(yl)[inside] - ry[inside]) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ry[inside])).all()
    past = np.abs(ry) > 2.0 ** 128
    assert past.any() and np.array_equal(_wide(yl)[past], np.sign(ry[past]) * np.inf)
