"""The head loss on the GPU where a loss is small at any size of the logits, where
weights are large, and through every tile height of each format.  Oracle and bounds:
tests/test_gpu_head.py."""

import numpy as np
import pytest
import torch

from gpu_util import banner, dev_bf16, dev_f32, host, require_gpu
from test_gpu_head import _bf16, _compare, _dev, _head, _labels, _poisoned, _wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [40, 300, 3500])
def test_small_losses_at_any_logit(V):
    """A row's logits are a, its label's a + b (whole numbers, exact in fp32), so that its
    loss is log1p((V - 1) e^-b) whatever a is, down to 1e-15 and below.  In powers of two a
    and a + b are off by 1.5 2^-24 of themselves (product and constant), both again by
    2^-18 less their cell, exponentials and sums (at most V / 4 + 64 terms in a chain) by 2^-22 +
    (V / 4 + 64) 2^-24: a relative error of loss and gradient."""
    q = require_gpu()
    banner(f"head small losses V={V}")
    levels = np.array([-100, -88, -64, -60, -45, -44, -36, -31, -29, -27, -10, 0, 10, 28, 44, 45, 60, 64, 88, 100.0])
    gaps = np.array([1, 2, 4, 7, 10, 14, 18, 20, 25, 30, 36.0])
    a, b = (x.reshape(-1) for x in np.meshgrid(levels, gaps, indexing="ij"))
    T, H, label = len(a), 64, 7
    X, W = np.zeros((T, H)), np.zeros((V, H))
    X[:, 0], X[:, 1] = a, b
    W[:, 0] = 1
    W[label, 1] = 1
    X = torch.from_numpy(X).to(torch.bfloat16).cuda()
    W = torch.from_numpy(W).to(torch.bfloat16).cuda()
    y, g = np.full(T, label), np.ones(T, dtype=np.float32)
    ref = np.log1p((V - 1) * np.exp(-b))
    rel = np.log(2) * (1.5 * 2.0 ** -24 * 1.4427 * (np.abs(a) + np.abs(a + b)) + 2.0 ** -17) + 2.0 ** -22 + (V / 4 + 64) * 2.0 ** -24
    loss, lse, dX = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g))
    for l, z in ((loss, lse), q.qlora_head_loss(W, X, _dev(y))):
        err = np.abs(host(l) / ref - 1)
        assert (err <= rel).all(), (a[err > rel], b[err > rel], host(l)[err > rel], ref[err > rel])
        rz = a + np.log(V - 1 + np.exp(b))
        assert (np.abs(host(z) - rz) <= 2.0 ** -20 * (1 + np.abs(rz))).all()
    # column 1: - (1 - p) of the label, rounded to bf16
    rest = -np.expm1(-ref)
    d1 = _wide(dX)[:, 1]
    assert (np.abs(-d1 / rest - 1) <= 2.0 ** -8 + 2 * rel).all()


def test_large_weights_with_a_gradient():
    """E, at most 2^64 a term, times weights of up to 2^39: rows of about 2^-36, whose
    largest logits are 40 to 142, in one cell and across its border, have finite gradients."""
    q = require_gpu()
    banner("head large weights")
    T, V, H = 40, 1300, 64
    W = torch.from_numpy(np.random.Generator(np.random.PCG64(3)).normal(0, 1, (V, H))).clamp(-3.9, 3.9).cuda()
    W = (W * 2.0 ** 37).to(torch.bfloat16)
    X = dev_bf16(_bf16(4, (T, H), 1.0)) * 2.0 ** -37 * 2
    X[::2] *= 2.0 ** 0.5 * 1.6
    Wv, y = _wide(W), _labels(5, T, V)
    g = np.ones(T, dtype=np.float32)
    loss, lse, dX = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, False, True))
    assert bool(torch.isfinite(dX).all()) and host(lse).max() > 44
    _compare(X, Wv, y, g, loss, lse, dX, whole=False)


# tests/test_head_shapes_cpu.py holds these to what they are for: each height of a tile of the logits
# and of dX, full and one row short of it and one past it, with more than one step of a
# product and a second column tile
LOGITS = [(T, 33024, 320) for T in (63, 65, 95, 97, 127, 129, 159, 161, 191, 193, 223, 225, 256, 257)]
GRADS = [(T, 3300, 16384) for T in (63, 65, 95, 97, 127, 129, 159, 161, 191, 193, 223)] + [(T, 4160, 16384) for T in (225, 256)]


@pytest.mark.parametrize("T,V,H", LOGITS + GRADS)
def test_16_bit_head_of_each_tile(T, V, H):
    q = require_gpu()
    banner(f"head tiles bf16 {T}x{V}x{H}")
    W, Wv = _head(q, "bf16", V + H, V, H, 4 / np.sqrt(H))
    X, y = dev_bf16(_bf16(V + 2, (T, H))), _labels(T, T, V)
    g = np.abs(np.random.Generator(np.random.PCG64(T)).normal(0, 1, T)).astype(np.float32)
    # the first and the last rows, and some of every 16 rows between
    rows = np.unique(np.concatenate([np.arange(0, 8), np.arange(0, T, 9), np.arange(T - 3, T)]))
    loss, lse, dX = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, False, True))
    _compare(X, Wv, y, g, loss, lse, dX, rows=rows)
    l2, z2 = q.qlora_head_loss(W, X, _dev(y), ws=_poisoned(q, T, V, H, False, False))
    _compare(X, Wv, y, g, l2, z2, rows=rows)
    # every row is the same row of a call of its own to within both calls' bounds
    d = (H / 16 + 16) * 2.0 ** -23 * (X.double().abs() @ W.double().abs().t().contiguous()).amax(1)
    for first in range(0, T, 32):
        part = slice(first, min(first + 32, T))
        lp, zp = q.qlora_head_loss(W, X[part].contiguous(), _dev(y[part]))
        slack = 2 * d[part] + 2.0 ** -18 * (1 + zp.abs())
        assert bool(((zp - lse[part]).abs() <= slack).all()) and bool(((lp - loss[part]).abs() <= 2 * slack).all())


@pytest.mark.parametrize("kind", ["nf4", "nodq", "fp8"])
@pytest.mark.parametrize("T,V,H", [(129, 33024, 320), (160, 33024, 320), (161, 33024, 320), (192, 33024, 320), (193, 33024, 320),
                                   (255, 33024, 320), (256, 32768, 320)])
def test_quantized_head_of_each_tile(kind, T, V, H):
    """The taller tiles of codes in more than one step of a product."""
    q = require_gpu()
    banner(f"head tiles {kind} {T}x{V}x{H}")
    W, Wv = _head(q, kind, V + H, V, H, 4 / np.sqrt(H))
    X, y = dev_bf16(_bf16(V + 2, (T, H))), _labels(T, T, V)
    g = np.abs(np.random.Generator(np.random.PCG64(T)).normal(0, 1, T)).astype(np.float32)
    rows = np.unique(np.concatenate([np.arange(0, 8), np.arange(0, T, 9), np.arange(T - 3, T)]))
    out = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, True, True))
    _compare(X, Wv, y, g, *out, rows=rows)
    _compare(X, Wv, y, g, *q.qlora_head_loss(W, X, _dev(y), ws=_poisoned(q, T, V, H, True, False)), rows=rows)
