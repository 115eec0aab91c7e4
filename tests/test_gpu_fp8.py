"""GPU parity of the 8-bit format and its linear layer against the fp64 oracle.

Codes, scales and dequantized weights are compared bit for bit.  Products:
  - pins: with one non-zero activation per row every sum has one term, so the
    result is a weight, exactly, at every k and n; with an identity weight it is
    the quantized activation, exactly;
  - Y and dX elsewhere: relative Frobenius <= 2e-3 (the rounding to bf16 is a
    half step, 2^-8 at most and 1.7e-3 in the mean square) and, for each
    element, 2^-8 of it (that half step) + 2^-12 of the sum of its terms'
    magnitudes (the matrix cores align the products of one instruction to about
    13 bits below the largest before they add them, 1.4e-4 < 2^-12 at worst
    over random codes; the adapter's hi + lo pairs are 2^-17 off);
  - dA, dB (fp32): 2e-5 relative Frobenius (each factor is a hi + lo pair, 2^-17
    at most, times fp32 sums)."""

import numpy as np
import pytest
import torch

import synth
from oracle import dense as odense
from oracle import fp8 as ofp8
from oracle import nf4 as onf4

from gpu_util import TOL, banner, dev_bf16, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu


def _bf16(seed, shape, std=1.0):
    return synth.bf16_bits(synth.normal_f32(seed, shape, std))


def _check(got_bits, ref, mag, what):
    got = onf4.bf16_bits_to_f32(got_bits).astype(np.float64)
    assert got.shape == ref.shape
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * mag
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])
    if ref.size >= 1024:  # fewer: the mean square of so few roundings says little
        assert odense.rel_frobenius(got, ref) <= TOL, what


def _rows(T, n=32):
    rng = np.random.Generator(np.random.PCG64(5))
    return np.unique(np.concatenate([[0, T - 1], rng.choice(T, size=min(n, T), replace=False)]))


# ------------------------------------------------------------------ format
@pytest.mark.parametrize("rows,cols", [(64, 64), (128, 128), (64, 192), (320, 64), (192, 4160), (1088, 448),
                                       (4096, 512)])
def test_quantize_dequantize_bit_exact(rows, cols):
    q = require_gpu()
    banner(f"fp8 quantize {rows}x{cols}")
    w = synth.normal_f32(rows + cols, (rows, cols), synth.W_STD)
    codes, scales = q.qlora_fp8_quantize(dev_f32(w))
    rc, rs = ofp8.quantize(w)
    assert np.array_equal(host(scales), rs)
    assert np.array_equal(host(codes), rc)
    wh = host_bits(q.qlora_fp8_dequantize(codes, scales, rows, cols))
    assert np.array_equal(wh, synth.bf16_bits(ofp8.dequantize(rc, rs).astype(np.float32)))


def test_quantize_edge_blocks():
    q = require_gpu()
    banner("fp8 edge blocks")
    w = np.zeros((128, 128 * 12), dtype=np.float32)
    rng = np.random.Generator(np.random.PCG64(7))
    blk = lambda i: w[:, 128 * i:128 * (i + 1)]
    blk(1)[:] = rng.normal(0, 1, (128, 128)) * 1e-39                      # subnormal weights
    blk(2)[:] = rng.normal(0, 1, (128, 128)) * 1e37
    blk(3)[3, 5] = 448.0
    blk(4)[3, 5] = np.nextafter(np.float32(448), np.float32(1000))
    blk(5)[:] = rng.uniform(-1, 1, (128, 128))
    blk(5)[0, 0] = 1.75                                                  # largest of its binade that fits
    blk(6)[0, 0] = np.float32(3.4028235e38)
    blk(7)[0, 0] = np.float32(1e-45)                                     # the smallest number
    mags = ofp8.e4m3_values()[:127]
    blk(8).reshape(-1)[:127] = mags
    blk(8).reshape(-1)[127:253] = -(mags[1:] + mags[:-1]) / 2            # ties
    blk(9)[:] = -0.0
    blk(10)[:] = np.where(rng.random((128, 128)) < 0.5, np.float32(2.0 ** -119), 0)
    blk(11)[127, 127] = -1.0
    codes, scales = q.qlora_fp8_quantize(dev_f32(w))
    rc, rs = ofp8.quantize(w)
    assert np.array_equal(host(scales), rs)
    assert np.array_equal(host(codes), rc)
    wh = host_bits(q.qlora_fp8_dequantize(codes, scales, *w.shape))
    assert np.array_equal(wh, synth.bf16_bits(ofp8.dequantize(rc, rs).astype(np.float32)))


# ------------------------------------------------------------------ pins
@pytest.mark.parametrize("n_in,n_out", [(64, 64), (192, 128), (320, 448), (512, 192)])
def test_one_hot_rows_read_the_weight_exactly(n_in, n_out):
    q = require_gpu()
    banner(f"fp8 one-hot {n_in}x{n_out}")
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(11, (n_out, n_in), synth.W_STD)))
    wh = host_bits(q.qlora_fp8_dequantize(W.codes, W.scales, n_out, n_in))
    eye = torch.eye(n_in, dtype=torch.bfloat16, device="cuda")
    for T in (n_in, 17, 16, 3, 1):
        X = eye[n_in - T:].contiguous() if T <= n_in else eye
        Y = host_bits(q.qlora_fp8_linear_fwd(W, X, None, None, 0, 0.0))
        assert np.array_equal(Y & 0x7fff, wh.T[n_in - X.shape[0]:] & 0x7fff)
    eye = torch.eye(n_out, dtype=torch.bfloat16, device="cuda")
    for T in (n_out, 33, 5, 1):
        dY = eye[n_out - T:].contiguous() if T <= n_out else eye
        dX, dA, dB = q.qlora_fp8_linear_bwd(W, None, dY, None, None, 0, 0.0)
        assert dA is None and dB is None
        assert np.array_equal(host_bits(dX) & 0x7fff, wh[n_out - dY.shape[0]:] & 0x7fff)


@pytest.mark.parametrize("T", [1, 5, 16, 40, 200])
def test_identity_weight_shows_the_quantized_rows(T):
    q = require_gpu()
    banner(f"fp8 identity T={T}")
    n = 448
    x = synth.normal_f32(21, (T, n), 1.0) * np.exp2(np.arange(n) % 40 - 20).astype(np.float32)
    x[0, :128] = 0.0
    if T > 4:
        x[1] *= np.float32(1e-36)
        x[2] *= np.float32(1e30)
        x[3] = 0.0
        x[4, 130] = -1.75
        x[4, 128:130] = 0
    bits = synth.bf16_bits(x)
    ref = synth.bf16_bits(ofp8.quantized_rows(odense.widen(bits)).astype(np.float32))
    W = q.qlora_fp8_quantize_weight(torch.eye(n, device="cuda"))
    Y = host_bits(q.qlora_fp8_linear_fwd(W, dev_bf16(bits), None, None, 0, 0.0))
    assert np.array_equal(Y & 0x7fff, ref & 0x7fff)
    dX, _, _ = q.qlora_fp8_linear_bwd(W, None, dev_bf16(bits), None, None, 0, 0.0)
    assert np.array_equal(host_bits(dX) & 0x7fff, ref & 0x7fff)


# ------------------------------------------------------------------ products
@pytest.mark.parametrize("T,n_in,n_out,r,alpha", [
    (1, 64, 64, 0, 0.0), (1, 4096, 1024, 16, 32.0), (2, 320, 192, 4, 8.0), (5, 192, 64, 256, 32.0),
    (16, 1024, 512, 64, 128.0), (17, 448, 320, 1, 2.0), (31, 576, 640, 24, 48.0), (33, 4160, 1088, 16, 32.0),
    (63, 64, 4096, 8, 16.0), (64, 2048, 256, 0, 0.0), (127, 832, 384, 8, 16.0), (129, 512, 128, 65, 32.0),
    (300, 4160, 1088, 0, 0.0), (515, 1024, 1472, 16, 32.0), (4096, 1088, 4160, 64, 128.0),
    (4109, 960, 4096, 8, 16.0), (4100, 4160, 320, 24, 48.0), (4096, 4096, 576, 0, 0.0),
])
def test_linear_matches_oracle(T, n_in, n_out, r, alpha):
    q = require_gpu()
    banner(f"fp8 linear T={T} in={n_in} out={n_out} r={r}")
    w = synth.normal_f32(31, (n_out, n_in), synth.W_STD)
    X, dY = _bf16(32, (T, n_in)), _bf16(33, (T, n_out))
    A, B = _bf16(34, (max(r, 1), n_in), 1.0 / n_in ** 0.5), _bf16(35, (n_out, max(r, 1)), 0.05)
    W = q.qlora_fp8_quantize_weight(dev_f32(w))
    Ad, Bd = (dev_bf16(A), dev_bf16(B)) if r else (None, None)
    Xd, dYd = dev_bf16(X), dev_bf16(dY)
    big = torch.full((T + 3, n_out), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = q.qlora_fp8_linear_fwd(W, Xd, Ad, Bd, r, alpha, Y=big[:T])
    assert bool((big[T:] == 7.0).all())  # rows behind the last are left alone
    dX, dA, dB = q.qlora_fp8_linear_bwd(W, Xd if r else None, dYd, Ad, Bd, r, alpha)
    Y, dX = host_bits(Y), host_bits(dX)

    Wh = ofp8.dequantize(*ofp8.quantize(w))
    rows = _rows(T)
    Xw, Gw, Aw, Bw = (odense.widen(t) for t in (X, dY, A, B))
    s = alpha / r if r else 0.0
    ref = ofp8.linear_fwd(Wh, Xw[rows], Aw, Bw, r, alpha)
    mag = np.abs(Xw[rows]) @ np.abs(Wh.T) + abs(s) * (np.abs(Xw[rows]) @ np.abs(Aw.T)) @ np.abs(Bw.T)
    _check(Y[rows], ref, mag, "Y")
    ref_dx, _, _ = ofp8.linear_bwd(Wh, Xw[rows], Gw[rows], Aw, Bw, r, alpha)
    mag = np.abs(Gw[rows]) @ np.abs(Wh) + abs(s) * (np.abs(Gw[rows]) @ np.abs(Bw)) @ np.abs(Aw)
    _check(dX[rows], ref_dx, mag, "dX")
    if r:
        V, U = Gw @ Bw, Xw @ Aw.T
        assert odense.rel_frobenius(host(dA), s * (V.T @ Xw)) <= 2e-5
        assert odense.rel_frobenius(host(dB), s * (Gw.T @ U)) <= 2e-5


@pytest.mark.parametrize("T,n_in,n_out,r,alpha", [
    (3, 8192, 64, 16, 32.0), (16, 8256, 192, 0, 0.0), (1, 14336, 128, 16, 32.0), (9, 8256, 64, 100, 50.0),
    (2, 4160, 4224, 256, 16.0), (13, 64, 8192, 100, 20.0), (16, 8192, 8256, 12, 24.0), (65, 2048, 192, 16, 32.0),
    (40, 14336, 64, 130, 65.0), (600, 2048, 4160, 0, 0.0), (1030, 1984, 2112, 100, 50.0), (96, 1920, 320, 256, 16.0),
    (64, 4096, 320, 16, 32.0), (192, 2048, 576, 8, 16.0), (256, 1024, 4160, 0, 0.0), (257, 1024, 448, 24, 48.0),
])
def test_linear_where_the_kernels_change(T, n_in, n_out, r, alpha):
    """Sizes next to which another kernel, tile or K split takes over."""
    test_linear_matches_oracle(T, n_in, n_out, r, alpha)


def test_empty_calls():
    q = require_gpu()
    banner("fp8 T = 0")
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(1, (64, 128), synth.W_STD)))
    X, dY = (torch.empty(0, n, dtype=torch.bfloat16, device="cuda") for n in (128, 64))
    A, B = dev_bf16(_bf16(2, (4, 128))), dev_bf16(_bf16(3, (64, 4)))
    assert q.qlora_fp8_linear_fwd(W, X, A, B, 4, 8.0).shape == (0, 64)
    dA, dB = torch.full((4, 128), 3.0, device="cuda"), torch.full((64, 4), 3.0, device="cuda")
    q.qlora_fp8_linear_bwd(W, X, dY, A, B, 4, 8.0, dA=dA, dB=dB)
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("T", [1, 4, 40, 300])
def test_a_row_that_is_not_finite_stays_its_own(T):
    q = require_gpu()
    banner(f"fp8 non-finite rows T={T}")
    n_in, n_out = 320, 192
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(41, (n_out, n_in), synth.W_STD)))
    X = dev_bf16(_bf16(42, (T, n_in)))
    clean = q.qlora_fp8_linear_fwd(W, X, None, None, 0, 0.0)
    bad = X.clone()
    bad[0, 5] = float("nan")
    if T > 3:
        bad[2, 300] = float("-inf")
    Y = q.qlora_fp8_linear_fwd(W, bad, None, None, 0, 0.0)
    hit = torch.isnan(bad).any(1) | torch.isinf(bad).any(1)
    assert bool(torch.isnan(Y[hit]).all())
    assert torch.equal(Y[~hit], clean[~hit])


@pytest.mark.parametrize("T", [1, 16, 300])
def test_repeated_streams_and_graphs(T):
    q = require_gpu()
    banner(f"fp8 repeat / stream / graph T={T}")
    n_in, n_out, r, alpha = 1024, 576, 16, 32.0
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(51, (n_out, n_in), synth.W_STD)))
    A, B = dev_bf16(_bf16(52, (r, n_in), 0.03)), dev_bf16(_bf16(53, (n_out, r), 0.05))
    X, dY = dev_bf16(_bf16(54, (T, n_in))), dev_bf16(_bf16(55, (T, n_out)))

    def both():
        return (q.qlora_fp8_linear_fwd(W, X, A, B, r, alpha), *q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, alpha))
    ref = [t.clone() for t in both()]
    assert all(torch.equal(a, b) for a, b in zip(both(), ref))
    need = max(q.qlora_fp8_workspace_bytes(T, n_in, n_out, r, b) for b in (False, True))
    for fill in (0x00, 0xff):  # workspace contents change nothing
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got = (q.qlora_fp8_linear_fwd(W, X, A, B, r, alpha, ws=ws),
               *q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, alpha, ws=ws))
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    keep = X.clone()
    X2 = dev_bf16(_bf16(56, (T, n_in)))
    for turn in range(3):
        X.copy_(X2 if turn == 1 else keep)
        want = [t.clone() for t in both()]  # eager work between the replays
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn


def test_binding_refuses_wrong_tensors():
    q = require_gpu()
    banner("fp8 binding refusals")
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(57, (128, 192), synth.W_STD)))
    A, B = dev_bf16(_bf16(58, (8, 192))), dev_bf16(_bf16(59, (128, 8)))
    X, dY = dev_bf16(_bf16(60, (40, 192))), dev_bf16(_bf16(61, (40, 128)))
    ok = q.qlora_fp8_linear_fwd(W, X, A, B, 8, 16.0)

    def refused(error, fn, *args, **kw):
        with pytest.raises(error):
            fn(*args, **kw)
    fwd, bwd = q.qlora_fp8_linear_fwd, q.qlora_fp8_linear_bwd
    refused(ValueError, fwd, W, dY, A, B, 8, 16.0)                                 # another width
    refused(ValueError, fwd, W, dev_bf16(_bf16(60, (192, 40))).t(), A, B, 8, 16.0)  # strided
    refused(ValueError, fwd, W, X.cpu(), A, B, 8, 16.0)                            # another device
    refused(ValueError, fwd, W, X, A[:4], B, 8, 16.0)                              # another rank
    refused(TypeError, fwd, W, X.half(), A, B, 8, 16.0)
    refused(TypeError, fwd, W, X, A, B, 8, 16.0, Y=torch.empty(40, 128, device="cuda"))
    refused(ValueError, fwd, W, X, A, B, 8, 16.0, Y=torch.empty(39, 128, dtype=torch.bfloat16, device="cuda"))
    refused(ValueError, bwd, W, X[:39], dY, A, B, 8, 16.0)
    refused(TypeError, bwd, W, X, dY, A, B, 8, 16.0, dA=torch.empty(8, 192, dtype=torch.bfloat16, device="cuda"))
    refused(q.QloraError, fwd, W, X, A, B, 8, float("nan"))
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    refused(q.QloraError, fwd, W, X, A, B, 8, 16.0, ws=small)
    refused(q.QloraError, bwd, W, X, dY, A, B, 8, 16.0, ws=small)
    refused(ValueError, fwd, W, X, A, B, 8, 16.0, ws=small.cpu())
    # views are at home as long as they are whole rows, 16-byte aligned
    big = torch.cat([X, X])
    assert torch.equal(fwd(W, big[40:], A, B, 8, 16.0), ok)
    odd = torch.empty(40 * 192 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(40, 192)
    refused(q.QloraError, fwd, W, odd, A, B, 8, 16.0)
    assert torch.equal(fwd(W, X, A, B, 8, 16.0), ok)


@pytest.mark.parametrize("T", [13, 300])
def test_gradients_are_the_differences_of_the_forward(T):
    """dA and dB against central differences of sum(dY * Y) over the kernel's
    own forward.  Y is linear in A and in B, so the only errors are Y's
    rounding (at most 2^-8 of each value, independent of one another: their
    sum's standard deviation is at most that times the norm) over the step, and
    the gradients' own."""
    q = require_gpu()
    banner(f"fp8 differences T={T}")
    n_in, n_out, r, alpha = 320, 192, 8, 16.0
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(62, (n_out, n_in), synth.W_STD)))
    A, B = dev_bf16(_bf16(63, (r, n_in), 0.5)), dev_bf16(_bf16(64, (n_out, r), 0.5))
    X, dY = dev_bf16(_bf16(65, (T, n_in))), dev_bf16(_bf16(66, (T, n_out)))
    _, dA, dB = q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, alpha)

    def loss(A, B):
        Y = q.qlora_fp8_linear_fwd(W, X, A, B, r, alpha)
        return (Y.double() * dY.double()).sum().item(), (Y.double() * dY.double()).norm().item()
    step = 0.5  # a power of two: A +- step is exact for |A| in [2^-2, 2)
    for P, grad, which in ((A, dA, 0), (B, dB, 1)):
        at = [(i, j) for i, j in ((0, 0), (P.shape[0] - 1, P.shape[1] - 1), (P.shape[0] // 2, 3))]
        for i, j in at:
            P0 = P.clone()
            P0[i, j] = 1.0  # Y is linear in this value, the gradient does not depend on it
            up, down = P0.clone(), P0.clone()
            up[i, j], down[i, j] = 1.0 + step, 1.0 - step
            (lu, nu), (ld, nd) = (loss(up, B), loss(down, B)) if which == 0 else (loss(A, up), loss(A, down))
            g = q.qlora_fp8_linear_bwd(W, X, dY, *((P0, B) if which == 0 else (A, P0)), r, alpha)[1 + which][i, j].item()
            bound = 5 * 2.0 ** -8 * (nu + nd) / (2 * step) + 1e-4 * abs(g)
            assert abs((lu - ld) / (2 * step) - g) <= bound, (which, i, j, (lu - ld) / (2 * step), g, bound)
