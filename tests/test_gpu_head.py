"""Cross entropy through an output head on the GPU against oracle/head.py in 64
bits.

Tolerances.  A logit sums H exact products of bf16 values in fp32, 16 in one matrix
instruction, H / 16 of those in a chain; with at most a whole step of 2^-23 a link it is
off by at most d = (H / 16 + 16) 2^-23 sum |x w|.  lse is a mean of logits plus 2^-22
of its parts: d + 2^-20 (1 + |lse|); a loss twice that.  dX's terms have weights that are off by 2 d
(as exponents), by 2^-8 (rounded to bf16) and 2^-18 (sums, exponentials), and dX itself by
2^-8: 2^-8 |dX| + (2^-8 + 2 d + 2^-17) mag, mag the sum of the terms' magnitudes.  That bound
goes with 1 - p of a row that is nearly sure.  2 d stands for e^(2 d) - 1, which is more where
logits are so large that d is no longer small: a weight p is then off by p (e^(2 d) - 1), but by
no more than 1, and rows with d > 1/64 get the sum of min(1, p (e^(2 d) - 1)) |W| in the place of
2 d mag.  Over a whole output errors are far smaller:
relative Frobenius 2e-5 for loss and lse; for dX 2.5e-3 (one rounding to bf16 is 1.7e-3, and
where one term is nearly all of the sum its own rounding adds as much: 1.7e-3 sqrt 2)."""

import numpy as np
import pytest
import torch

import synth
from oracle import dense as odense
from oracle import fp8 as ofp8
from oracle import head as ohead
from oracle import nf4 as onf4

from gpu_util import banner, dev_bf16, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu


def _bf16(seed, shape, std=1.0):
    return synth.bf16_bits(synth.normal_f32(seed, shape, std))


def _wide(t):
    return onf4.bf16_bits_to_f32(host_bits(t)).astype(np.float64)


def _head(q, kind, seed, V, H, std):
    """(the head as the call takes it, its values in 64 bits)."""
    w = synth.normal_f32(seed, (V, H), std)
    if kind == "bf16":
        t = dev_bf16(synth.bf16_bits(w))
        return t, _wide(t)
    if kind == "fp8":
        W = q.qlora_fp8_quantize_weight(dev_f32(w))
        return W, ofp8.dequantize(host(W.codes), host(W.scales))
    if kind == "nf4":
        W = q.nf4_quantize_weight(dev_f32(w))
        v = q.nf4_dequantize(W.codes, W.absmax_q, W.absmax_scale, V * H)
    else:
        W = q.nf4_quantize_weight_nodq(dev_f32(w))
        v = q.nf4_dequantize_nodq(W.codes, W.absmax_scale, V * H)
    return W, _wide(v).reshape(V, H)


def _labels(seed, T, V):
    y = np.random.Generator(np.random.PCG64(seed)).integers(0, V, T)
    if T > 4:
        y[1], y[3], y[T - 1] = -100, V, 0
    if T > 8:
        y[4], y[5], y[6] = V - 1, np.iinfo(np.int64).max, np.iinfo(np.int64).min
    return y


def _dev(y):
    return torch.from_numpy(np.ascontiguousarray(y)).cuda()


def _compare(X, W, y, g, loss, lse, dX=None, rows=None, whole=True):
    """The outputs' rows (all, or some) against the oracle."""
    rows = np.arange(len(y)) if rows is None else rows
    X, y, g = _wide(X)[rows], y[rows], g[rows].astype(np.float64)
    rl, rz, rdX, _, mag = ohead.loss_grad(X, W, y, g)
    loss, lse = host(loss)[rows].astype(np.float64), host(lse)[rows].astype(np.float64)
    d = (X.shape[1] / 16 + 16) * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T).max(axis=1)
    assert (np.abs(lse - rz) <= d + 2.0 ** -20 * (1 + np.abs(rz))).all()
    assert (np.abs(loss - rl) <= 2 * d + 2.0 ** -19 * (1 + np.abs(rz))).all()
    assert not loss[~ohead.has_label(y, W.shape[0])].any()
    if whole:
        assert odense.rel_frobenius(lse, rz) <= 2e-5
        if rl.any():
            assert odense.rel_frobenius(loss, rl) <= 2e-5
    if dX is None:
        return
    dX = _wide(dX)[rows]
    bound = 2.0 ** -8 * np.abs(rdX) + (2.0 ** -8 + 2.0 ** -17) * mag + 1e-38
    for t in range(len(y)):
        if d[t] <= 1 / 64:
            bound[t] += (2 * d[t] + 4 * d[t] ** 2) * mag[t]
        elif ohead.has_label(y[t], W.shape[0]):
            logp = X[t] @ W.T - rz[t]
            grow = 2 * d[t] if d[t] > 300 else np.log(np.expm1(2 * d[t]))
            bound[t] += np.abs(g[t]) * (np.exp(np.minimum(0.0, logp + grow)) @ np.abs(W))
    assert (np.abs(dX - rdX) <= bound).all()
    if whole and rdX.any():
        assert odense.rel_frobenius(dX, rdX) <= 2.5e-3


def _poisoned(q, T, V, H, expand, grad):
    return torch.full((q.qlora_head_workspace_bytes(T, V, H, expand, grad),), 0xff, dtype=torch.uint8, device="cuda")


# every tile height next to its borders, vocabularies next to a tile's end, one and two columns of
# dX tiles, splits of the vocabulary with and without a rest, one token to many
SIZES = [(1, 1, 64), (1, 2, 64), (2, 63, 128), (1, 1000, 320), (7, 255, 64), (16, 256, 192), (33, 257, 256), (64, 700, 320),
         (65, 511, 64), (100, 1025, 576), (128, 513, 64), (129, 300, 128), (256, 2100, 192), (257, 777, 64), (300, 5003, 320),
         (520, 4099, 64), (3, 20000, 128), (40, 9000, 1088)]


@pytest.mark.parametrize("T,V,H", SIZES)
def test_loss_and_gradient(T, V, H):
    q = require_gpu()
    banner(f"head {T}x{V}x{H}")
    W, Wv = _head(q, "bf16", T + V + H, V, H, 4 / np.sqrt(H))
    X, y = dev_bf16(_bf16(V + 1, (T, H))), _labels(T + V, T, V)
    g = np.abs(synth.normal_f32(T, (T,), 1.0)) + 0.1
    g[T // 2] *= -1
    loss, lse, dX = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, False, True))
    _compare(X, Wv, y, g, loss, lse, dX)
    l2, z2 = q.qlora_head_loss(W, X, _dev(y), ws=_poisoned(q, T, V, H, False, False))
    _compare(X, Wv, y, g, l2, z2)
    again = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g))
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, lse, dX)))


@pytest.mark.parametrize("kind", ["nf4", "nodq", "fp8"])
@pytest.mark.parametrize("T,V,H", [(1, 64, 64), (5, 320, 128), (32, 704, 320), (33, 704, 320), (64, 1088, 192), (70, 1088, 192), (128, 704, 1088),
                                   (300, 704, 320), (512, 2112, 320), (513, 2112, 320)])
def test_quantized_heads(kind, T, V, H):
    q = require_gpu()
    banner(f"head {kind} {T}x{V}x{H}")
    W, Wv = _head(q, kind, V + H, V, H, 4 / np.sqrt(H))
    X, y = dev_bf16(_bf16(V + 2, (T, H))), _labels(T, T, V)
    g = np.abs(synth.normal_f32(T + 1, (T,), 1.0))
    out = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, True, True))
    _compare(X, Wv, y, g, *out)
    _compare(X, Wv, y, g, *q.qlora_head_loss(W, X, _dev(y), ws=_poisoned(q, T, V, H, True, False)))


@pytest.mark.parametrize("kind", ["nf4", "fp8"])
@pytest.mark.parametrize("T,V,H", [(256, 32768, 64), (160, 33024, 64), (192, 33024, 64), (250, 33024, 64), (250, 8256, 4160),
                                   (160, 4160, 16384), (190, 4160, 16384), (250, 4160, 16384)])
def test_quantized_heads_of_each_tile(kind, T, V, H):
    """Sizes that take each height of a tile of the logits (many vocabulary rows) and
    of dX (long rows), up to 512 rows in the weight's own format."""
    q = require_gpu()
    banner(f"head tiles {kind} {T}x{V}x{H}")
    W, Wv = _head(q, kind, V + H, V, H, 4 / np.sqrt(H))
    X, y = dev_bf16(_bf16(V + 2, (T, H))), _labels(T, T, V)
    g = np.abs(synth.normal_f32(T + 1, (T,), 1.0))
    rows = np.unique(np.concatenate([np.arange(0, 8), np.arange(0, T, 9), np.arange(T - 3, T)]))
    out = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, True, True))
    _compare(X, Wv, y, g, *out, rows=rows)
    _compare(X, Wv, y, g, *q.qlora_head_loss(W, X, _dev(y), ws=_poisoned(q, T, V, H, True, False)), rows=rows)


def test_vocabulary_in_pieces_16_bit():
    """4096 rows and 70001 columns: three pieces, a last one that ends inside a
    tile; rows in one round, then 4100 rows in two (with fewer pieces)."""
    q = require_gpu()
    V, H = 70001, 64
    W, Wv = _head(q, "bf16", 5, V, H, 0.5)
    for T in (4096, 4100):
        banner(f"head pieces {T}x{V}x{H}")
        X, y = dev_bf16(_bf16(6, (T, H))), _labels(7, T, V)
        y[10:16] = 23551, 23552, 35071, 35072, 47104, V - 1  # next to where pieces meet
        g = np.abs(synth.normal_f32(8, (T,), 1.0))
        out = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, False, True))
        rows = np.concatenate([np.arange(0, 20), np.arange(2040, 2060), np.arange(T - 30, T)])
        _compare(X, Wv, y, g, *out, rows=rows)
        _compare(X, Wv, y, g, *q.qlora_head_loss(W, X, _dev(y)), rows=rows)


@pytest.mark.parametrize("kind", ["nf4", "nodq", "fp8"])
def test_vocabulary_in_pieces_quantized(kind):
    """Rows of 16384 columns: 520 of them make pieces of at most 2^27 weights, two of 4352
    and 3904 rows of the head; 128-row blocks and 16384-weight groups begin anew in each
    piece.  Three rows take the weight as it is, in one piece."""
    q = require_gpu()
    V, H = 8256, 16384
    W, Wv = _head(q, kind, 9, V, H, 0.03)
    for T in (3, 520):
        banner(f"head pieces {kind} {T}x{V}x{H}")
        X, y = dev_bf16(_bf16(10, (T, H))), np.resize(np.array([4351, 4352, 8255]), T)
        g = np.resize(np.array([1.0, -2.0, 0.5], dtype=np.float32), T)
        rows = np.unique(np.concatenate([np.arange(3), np.arange(T - 3, T)]))
        _compare(X, Wv, y, g, *q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, True, True)), rows=rows)
        _compare(X, Wv, y, g, *q.qlora_head_loss(W, X, _dev(y)), rows=rows)


@pytest.mark.parametrize("kind", ["nf4", "nodq", "fp8"])
def test_long_vocabulary_in_its_own_format(kind):
    """512 rows and 262464 columns are two pieces with a gradient, both read as codes."""
    q = require_gpu()
    T, V, H = 512, 262144 + 320, 64
    banner(f"head codes in pieces {kind}")
    W, Wv = _head(q, kind, 51, V, H, 0.5)
    X, y = dev_bf16(_bf16(52, (T, H))), _labels(53, T, V)
    y[10:16] = 131071, 131072, 131327, 131328, 262143, V - 1
    g = np.abs(synth.normal_f32(54, (T,), 1.0))
    rows = np.concatenate([np.arange(0, 20), np.arange(T - 4, T)])
    _compare(X, Wv, y, g, *q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, True, True)), rows=rows)
    _compare(X, Wv, y, g, *q.qlora_head_loss(W, X, _dev(y), ws=_poisoned(q, T, V, H, True, False)), rows=rows)


@pytest.mark.parametrize("T", [96, 48])
@pytest.mark.parametrize("size", [30.0, 100.0, 400.0, 3000.0, 1e6, 1e30])
def test_logits_of_any_size(size, T):
    """Rows whose logits spread over +-size: their tiles, pieces and label lie in
    different powers of 2^128.  The first column tile holds the smaller logits for
    half of the rows and the larger for the others."""
    q = require_gpu()
    banner(f"head logits of {size}")
    V, H = 1300, 64
    W, _ = _head(q, "bf16", 11, V, H, 0.5)
    W[:256] *= 0.125
    W[1290:] *= 2
    Wv = _wide(W)
    X = dev_bf16(_bf16(12, (T, H))) * (size / 8)
    X[::2] = X[::2] / 64
    X[5] = -X[5]
    y = _labels(13, T, V)
    y[20:30] = np.argmax(_wide(X)[20:30] @ Wv.T, axis=1)   # surest
    y[30:40] = np.argmin(_wide(X)[30:40] @ Wv.T, axis=1)   # as wrong as can be
    y[40:44] = np.arange(4)
    g = np.ones(T, dtype=np.float32)
    loss, lse, dX = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, False, True))
    _compare(X, Wv, y, g, loss, lse, dX, whole=size < 1e3)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(dX).all())


def test_cells_across_pieces():
    """Three pieces of the vocabulary whose logits rise by more than a cell from
    one to the next (what was accumulated shrinks to nothing or by 2^-128), fall, or lie on
    both sides of a cell's border (64 in powers of two)."""
    q = require_gpu()
    banner("head cells across pieces")
    T, V, H = 4096, 70000, 64
    W = dev_bf16(_bf16(14, (V, H), 0.05))
    W[:, 0] = 0
    W[16000:16010, 0] = 1
    W[30000:30010, 0] = 2
    W[60000:60010, 0] = 4
    W[300:303, 1] = 8
    Wv = _wide(W)
    X = dev_bf16(_bf16(15, (T, H), 0.5))
    a = torch.linspace(-400, 400, T, device="cuda")
    X[:, 0] = a.to(torch.bfloat16)
    X[:, 1] = 0
    X[1000:1100, 1] = 44.0 / 8      # logits of 44: powers of two of 63.5
    X[1100:1200, 1] = 44.75 / 8     # 64.6
    y = _labels(16, T, V)
    y[2000:2020] = 30000
    y[2020:2040] = 60003
    y[3000:3040] = 16003
    y[1000:1020] = 301
    g = np.ones(T, dtype=np.float32)
    out = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g), ws=_poisoned(q, T, V, H, False, True))
    rows = np.concatenate([np.arange(0, 40), np.arange(990, 1030), np.arange(1090, 1130), np.arange(1990, 2110, 3),
                           np.arange(3000, 3050, 2), np.arange(T - 30, T)])
    _compare(X, Wv, y, g, *out, rows=rows, whole=False)
    _compare(X, Wv, y, g, *q.qlora_head_loss(W, X, _dev(y)), rows=rows, whole=False)


def test_small_gradients_keep_their_digits():
    """Rows that are sure of their label up to 1 - p of 1e-2 .. 1e-12: the gradient
    is right in relation to 1 - p (the bound of _compare does that), and so is the
    loss: relative 1e-4 (the logits' own error, 1e-5 absolute, as an exponent)."""
    q = require_gpu()
    banner("head sure rows")
    T, V, H = 64, 3000, 256
    W, Wv = _head(q, "bf16", 17, V, H, 0.25)
    y = np.random.Generator(np.random.PCG64(18)).integers(0, V, T)
    sure = np.linspace(14, 36, T)[:, None] / (Wv[y] ** 2).sum(axis=1, keepdims=True)
    X = dev_bf16(synth.bf16_bits((0.2 * synth.normal_f32(19, (T, H), 1.0) + sure * Wv[y]).astype(np.float32)))
    g = np.ones(T, dtype=np.float32)
    loss, lse, dX = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(g))
    _compare(X, Wv, y, g, loss, lse, dX, whole=False)
    rl, _, rdX, rest, _ = ohead.loss_grad(_wide(X), Wv, y, g.astype(np.float64))
    assert rest.min() < 1e-9 and rest.max() > 1e-4
    assert (np.abs(host(loss) / rl - 1) <= 1e-4).all()
    err = np.linalg.norm(_wide(dX) - rdX, axis=1) / np.linalg.norm(rdX, axis=1)
    assert err.max() <= 1e-2


def test_rows_that_are_not_finite_stay_alone():
    q = require_gpu()
    banner("head not finite")
    T, V, H = 70, 600, 128
    W, Wv = _head(q, "bf16", 21, V, H, 0.3)
    X, y = dev_bf16(_bf16(22, (T, H))), _labels(23, T, V)
    g = dev_f32(np.ones(T))
    clean = q.qlora_head_loss_grad(W, X, _dev(y), g)
    bad = X.clone()
    bad[2, 3], bad[20, 0], bad[40, 127] = float("nan"), float("inf"), float("-inf")
    bad[1, 0] = float("nan")  # a row without a label
    loss, lse, dX = q.qlora_head_loss_grad(W, bad, _dev(y), g)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    for t in (1, 2, 20, 40):
        keep[t] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip((loss, lse, dX), clean))
    for t in (2, 20, 40):
        assert bool(torch.isnan(loss[t])) and bool(torch.isnan(lse[t])) and bool(torch.isnan(dX[t]).all())
    assert loss[1] == 0 and not dX[1].any() and bool(torch.isnan(lse[1]))
    # columns of -inf count for nothing: the logits of the row that meets them
    W2 = W.clone()
    W2[7], W2[300:310] = 0, 0
    W2[7, 0], W2[300:310, 0] = float("-inf"), float("-inf")
    X2 = X.clone()
    X2[:, 0] = X[:, 0].abs() + 0.25
    y2 = np.where(y == 7, 8, y)
    y2 = np.where((y2 >= 300) & (y2 < 310), 8, y2)
    loss, lse, _ = q.qlora_head_loss_grad(W2, X2, _dev(y2), g)
    live = np.ones(V, dtype=bool)
    live[7] = live[300:310] = False
    wl = _wide(W2)[live]
    ref, rz = ohead.loss_grad(_wide(X2), wl, np.where(ohead.has_label(y2, V), np.cumsum(live)[np.clip(y2, 0, V - 1)] - 1, -1))
    assert np.allclose(host(loss), ref, atol=1e-4) and np.allclose(host(lse), rz, atol=1e-4)


def test_gradient_is_the_difference_of_the_loss():
    """dX against central differences of the call's own loss along a direction:
    the loss is smooth; step h = 2^-4 gives h^2 |f'''| / 6 <= 1e-3 here, the loss's
    own error 1e-5 / h."""
    q = require_gpu()
    banner("head differences")
    T, V, H = 20, 500, 128
    W, _ = _head(q, "bf16", 25, V, H, 0.1)
    y = np.random.Generator(np.random.PCG64(26)).integers(0, V, T)
    X = torch.round(dev_bf16(_bf16(27, (T, H))).float() * 16) / 16  # X +- h exact in bf16
    X = X.clamp(-7, 7).to(torch.bfloat16)
    dX = q.qlora_head_loss_grad(W, X, _dev(y), dev_f32(np.ones(T)))[2]
    h = 2.0 ** -4
    for j in (0, 55, 127):
        up, dn = X.clone(), X.clone()
        up[:, j] += h
        dn[:, j] -= h
        assert torch.equal((up[:, j].float() - dn[:, j].float()), torch.full((T,), 2 * h, device="cuda"))
        diff = (q.qlora_head_loss(W, up, _dev(y))[0] - q.qlora_head_loss(W, dn, _dev(y))[0]) / (2 * h)
        assert bool(((diff - dX[:, j].float()).abs() <= 2.0 ** -8 * dX[:, j].float().abs() + 5e-4).all())


@pytest.mark.parametrize("kind,T", [("bf16", 40), ("bf16", 300), ("fp8", 300), ("nf4", 20), ("fp8", 100), ("nf4", 600)])
def test_streams_and_graphs(kind, T):
    q = require_gpu()
    banner(f"head streams and graphs {kind} T={T}")
    V, H = 2112, 320
    W, _ = _head(q, kind, 31, V, H, 0.2)
    X, y, g = dev_bf16(_bf16(32, (T, H))), _dev(_labels(33, T, V)), dev_f32(np.ones(T) / T)

    def both():
        return (*q.qlora_head_loss_grad(W, X, y, g), *q.qlora_head_loss(W, X, y))
    ref = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = both()
        graphs.append((gr, out))
    keep, other = X.clone(), dev_bf16(_bf16(34, (T, H), 3.0))
    for turn in range(3):
        X.copy_(other if turn == 1 else keep)
        want = [t.clone() for t in both()]
        for gr, out in graphs:
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn


def test_slices_of_longer_vectors():
    """labels shifted by one in front of their rows, as a causal model's are, and the
    other vectors at odd elements: the bits of the call on copies."""
    q = require_gpu()
    banner("head slices")
    T, V, H = 37, 2112, 320
    W, _ = _head(q, "bf16", 41, V, H, 0.2)
    X, y, g = dev_bf16(_bf16(42, (T + 1, H))), _dev(_labels(43, T + 1, V)), dev_f32(np.linspace(0.5, 1, T + 1).astype(np.float32))
    got = q.qlora_head_loss_grad(W, X[:-1], y[1:], g[1:])
    want = q.qlora_head_loss_grad(W, X[:-1].clone(), y[1:].clone(), g[1:].clone())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(q.qlora_head_loss(W, X[:-1], y[1:]), want))


def test_loss_in_pieces_16_bit():
    """4096 rows and 2^21 + 300 columns are two pieces without a gradient; sixteen of the
    rows are one.  A sum of positive terms is off by at most its longest chain times
    2^-24: 16 terms a lane, 5 more over the wave, 16400 blocks by 16 waves and their 16
    sums, 1063 in all: 6.4e-5 of the sum and as much of lse, twice that between two calls."""
    q = require_gpu()
    banner("head loss in pieces")
    T, V, H = 4096, (1 << 21) + 300, 64
    torch.manual_seed(5)
    W = torch.randn(V, H, device="cuda").to(torch.bfloat16)
    X = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    y = torch.randint(0, V, (T,), device="cuda")
    y[::5], y[1] = -100, V - 1
    loss, lse = q.qlora_head_loss(W, X, y)
    rows = torch.arange(0, T, 256, device="cuda")
    rows[0] = 1
    one, base = q.qlora_head_loss(W, X[rows].contiguous(), y[rows])
    assert (lse[rows] - base).abs().max() <= 1.3e-4 and (loss[rows] - one).abs().max() <= 1.3e-4
    logits = (X[1].double() * W.double()).sum(-1)
    assert abs(lse[1].item() - torch.logsumexp(logits, 0).item()) <= 1e-4
    assert abs(loss[1].item() - (torch.logsumexp(logits, 0) - logits[-1]).item()) <= 1e-4


def test_empty_and_refusals():
    q = require_gpu()
    banner("head T=0 and refusals")
    W = torch.zeros(10, 64, dtype=torch.bfloat16, device="cuda")
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse, dX = q.qlora_head_loss_grad(W, X, y, torch.empty(0, device="cuda"))
    assert loss.shape == lse.shape == (0,) and dX.shape == (0, 64)
    X, y, g = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")

    def refused(error, *args, **kw):
        with pytest.raises(error):
            q.qlora_head_loss_grad(*args, **kw)
    refused(TypeError, W, X, y.int(), g)
    refused(TypeError, W.float(), X, y, g)
    refused(ValueError, W[:, :32].contiguous(), X, y, g)
    refused(ValueError, W.t().contiguous().t(), X, y, g)
    refused(ValueError, W, X, y[:3], g)
    refused(ValueError, W, X, y, g.cpu())
    refused(ValueError, W, X, y, g, dX=torch.empty(64, 4, dtype=torch.bfloat16, device="cuda"))
    refused(q.QloraError, W, X, y, g, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    refused(q.QloraError, torch.zeros(10, 96, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 96, dtype=torch.bfloat16, device="cuda"), y, g)
