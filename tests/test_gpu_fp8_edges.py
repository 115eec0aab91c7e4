"""The 8-bit linear layer where its inputs leave the ordinary (rows that are
not finite, adapter products past bf16's largest, transposed tensors), where
its products are exact, and with any contents of its workspace, on another
stream and in graphs, at sizes that split the sums.

Above 16 tokens sU and sV meet dB and dA as three bf16 parts, up to 16 as fp32
values: the relative Frobenius bound of 2e-5 in test_gpu_fp8.py has room for
two parts (2^-17), the one for exact values here has not."""

import numpy as np
import pytest
import torch

import synth
from oracle import dense as odense
from oracle import fp8 as ofp8
from oracle import nf4 as onf4

from gpu_util import banner, dev_bf16, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu


def _bf16(seed, shape, std=1.0):
    return synth.bf16_bits(synth.normal_f32(seed, shape, std))


def _wide(t):
    return onf4.bf16_bits_to_f32(host_bits(t)).astype(np.float64)


# the forward's and backward's routes: up to 16 tokens with U formed inside (r <= 16) and before
# (above), the GEMM's 32-, 64- and 128-row tiles, one of them with K split
ROUTES = [(2, 320, 192, 16), (16, 320, 192, 24), (40, 320, 192, 8), (40, 2048, 2112, 8), (200, 320, 192, 48),
          (300, 320, 192, 100)]


@pytest.mark.parametrize("T,n_in,n_out,r", ROUTES)
def test_adapter_products_past_bf16(T, n_in, n_out, r):
    """s X A^T meets the matrix cores as bf16 parts.  One of its values between
    bf16's largest and fp32's has to count as the finite number it is, an
    infinite one as infinite with its sign: what is left of an infinite part
    must not be inf - inf.

    Row 0 has one value, c 2^63 with c = 181/128, and A's rows c 2^64 there: s X
    A^T = 1.99957 2^127 with s = 1, exact in fp32, above bf16's largest (1.99219
    2^127) by more than the half step that rounds to it.  Row 1 gives 2^130,
    infinite.  B's first column is 2^-20, the rest 0, so that rank 0 alone
    counts in Y and dX; the other ranks' infinities meet zeros and are no part
    of this: their A is 0."""
    q = require_gpu()
    banner(f"fp8 adapter products past bf16 T={T} {n_in}x{n_out} r={r}")
    c = 181 / 128
    u = c * c * 2.0 ** 127
    assert (2 - 2.0 ** -8) * 2.0 ** 127 < u < np.finfo(np.float32).max
    W = q.qlora_fp8_quantize_weight(torch.zeros(n_out, n_in, device="cuda"))
    at = n_in // 2
    A = torch.zeros(r, n_in, dtype=torch.bfloat16, device="cuda")
    A[0, at] = c * 2.0 ** 64
    B = torch.zeros(n_out, r, dtype=torch.bfloat16, device="cuda")
    B[:, 0] = 2.0 ** -20
    X = torch.zeros(T, n_in, dtype=torch.bfloat16, device="cuda")
    X[0, at], X[1, at] = c * 2.0 ** 63, 2.0 ** 66
    Y = _wide(q.qlora_fp8_linear_fwd(W, X, A, B, r, float(r)))
    assert (np.abs(Y[0] - u * 2.0 ** -20) <= 2.0 ** -8 * u * 2.0 ** -20).all()
    assert np.isposinf(Y[1]).all() and not Y[2:].any()

    # dB = dY^T sU, first without the infinite row
    half = n_out // 2
    one = X.clone()
    one[1] = 0
    dY = torch.zeros(T, n_out, dtype=torch.bfloat16, device="cuda")
    dY[0] = 2.0 ** -20
    _, _, dB = q.qlora_fp8_linear_bwd(W, one, dY, A, B, r, float(r))
    dB = host(dB).astype(np.float64)
    assert (np.abs(dB[:, 0] / (u * 2.0 ** -20) - 1) <= 2.0 ** -22).all() and not dB[:, 1:].any()
    dY[1] = -1.0
    _, _, dB = q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, float(r))
    assert np.isneginf(host(dB)[:, 0]).all() and not host(dB)[:, 1:].any()

    # dA = sV^T X and dX = sV A, sV = s dY B: the same numbers on the other side
    B.zero_()
    B[half, 0] = c * 2.0 ** 64
    A.zero_()
    A[0] = 2.0 ** -20
    X.fill_(0)
    X[0], X[1] = 2.0 ** -20, -1.0
    dY.zero_()
    dY[0, half] = c * 2.0 ** 63
    dX, dA, _ = q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, float(r))
    assert (np.abs(_wide(dX)[0] - u * 2.0 ** -20) <= 2.0 ** -8 * u * 2.0 ** -20).all() and not _wide(dX)[1:].any()
    dA = host(dA).astype(np.float64)
    assert (np.abs(dA[0] / (u * 2.0 ** -20) - 1) <= 2.0 ** -22).all() and not dA[1:].any()
    dY[1, half] = 2.0 ** 66
    dX, dA, _ = q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, float(r))
    assert np.isposinf(_wide(dX)[1]).all() and not _wide(dX)[2:].any()
    assert np.isneginf(host(dA)[0]).all() and not host(dA)[1:].any()


def test_transposed_tensors_are_refused():
    """Contiguous tensors of the right element count in the other order; other
    views of the same rows stay at home."""
    q = require_gpu()
    banner("fp8 transposed tensors")
    T, n_in, n_out, r = 40, 192, 128, 8
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(301, (n_out, n_in), synth.W_STD)))
    X, dY = dev_bf16(_bf16(302, (T, n_in))), dev_bf16(_bf16(303, (T, n_out)))
    A, B = dev_bf16(_bf16(304, (r, n_in))), dev_bf16(_bf16(305, (n_out, r)))
    Y = q.qlora_fp8_linear_fwd(W, X, A, B, r, 16.0)
    grads = q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, 16.0)
    At, Bt = A.t().contiguous(), B.t().contiguous()
    turned = q.FP8Weight(W.codes.t().contiguous(), W.scales, n_out, n_in)
    for a, b, w in ((At, B, W), (A, Bt, W), (At, Bt, W), (A, B, turned)):
        with pytest.raises(ValueError):
            q.qlora_fp8_linear_fwd(w, X, a, b, r, 16.0)
        with pytest.raises(ValueError):
            q.qlora_fp8_linear_bwd(w, X, dY, a, b, r, 16.0)
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(W, X, A, B, r, 16.0, Y=torch.empty(n_out, T, dtype=torch.bfloat16, device="cuda"))
    flat = q.FP8Weight(W.codes.view(-1), W.scales.view(-1), n_out, n_in)
    deep = torch.empty(5, 8, n_out, dtype=torch.bfloat16, device="cuda")
    assert q.qlora_fp8_linear_fwd(flat, X, A[None], B.view(-1), r, 16.0, Y=deep) is deep
    assert torch.equal(deep.view(T, n_out), Y)
    assert all(torch.equal(a, b) for a, b in zip(q.qlora_fp8_linear_bwd(flat, X, dY, A[None], B.view(-1), r, 16.0), grads))


# ------------------------------------------------------------------ rows that are not finite
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T,n_in,n_out,r", ROUTES)
def test_a_row_that_is_not_finite_stays_its_own(T, n_in, n_out, r, bad):
    """With an adapter, forward and backward, what is not finite in X's row 1
    reaches that row of Y, one column of dA and, through U's row, all of dB; in
    dY's row 1 that row of dX, one row of dB and, through V's, all of dA.  The
    rest is the clean call's bit for bit."""
    q = require_gpu()
    banner(f"fp8 non-finite rows T={T} {n_in}x{n_out} r={r} {bad}")
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(311, (n_out, n_in), synth.W_STD)))
    X, dY = dev_bf16(_bf16(312, (T, n_in))), dev_bf16(_bf16(313, (T, n_out)))
    A, B = dev_bf16(_bf16(314, (r, n_in), n_in ** -0.5)), dev_bf16(_bf16(315, (n_out, r), 0.05))
    Y = q.qlora_fp8_linear_fwd(W, X, A, B, r, 2.0 * r)
    dX, dA, dB = q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, 2.0 * r)
    assert all(bool(torch.isfinite(t).all()) for t in (Y, dX, dA, dB))
    rest = torch.arange(T, device="cuda") != 1

    at = n_in - 59
    Xb = X.clone()
    Xb[1, at] = bad
    Yb = q.qlora_fp8_linear_fwd(W, Xb, A, B, r, 2.0 * r)
    assert bool(torch.isnan(Yb[1]).all()) and torch.equal(Yb[rest], Y[rest])
    dXb, dAb, dBb = q.qlora_fp8_linear_bwd(W, Xb, dY, A, B, r, 2.0 * r)
    cols = torch.arange(n_in, device="cuda") != at
    assert torch.equal(dXb, dX) and torch.equal(dAb[:, cols], dA[:, cols])
    assert not bool(torch.isfinite(dAb[:, at]).any()) and not bool(torch.isfinite(dBb).any())

    at = n_out - 59
    Gb = dY.clone()
    Gb[1, at] = bad
    dXb, dAb, dBb = q.qlora_fp8_linear_bwd(W, X, Gb, A, B, r, 2.0 * r)
    rows = torch.arange(n_out, device="cuda") != at
    assert bool(torch.isnan(dXb[1]).all()) and torch.equal(dXb[rest], dX[rest])
    assert torch.equal(dBb[rows], dB[rows])
    assert not bool(torch.isfinite(dBb[at]).any()) and not bool(torch.isfinite(dAb).any())


# ------------------------------------------------------------------ exact products
def _no_minus_zero(bits):
    return np.where(bits == 0x8000, 0, bits)


@pytest.mark.parametrize("n_in,n_out", [(192, 128), (320, 448), (512, 192)])
def test_one_hot_rows_read_the_weight_with_its_sign(n_in, n_out):
    """One value of +-1 a row: the product is a weight or its negative, all 16
    bits (a zero may have either sign)."""
    q = require_gpu()
    banner(f"fp8 signed one-hot {n_in}x{n_out}")
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(321, (n_out, n_in), synth.W_STD)))
    wh = host_bits(q.qlora_fp8_dequantize(W.codes, W.scales, n_out, n_in))
    assert ((wh & 0x8000) != 0).any() and ((wh & 0x8000) == 0).any()
    for n, ref in ((n_in, wh.T), (n_out, wh)):
        eye = torch.eye(n, dtype=torch.bfloat16, device="cuda")
        eye[::2] *= -1.0
        want = ref.copy()
        want[::2] ^= 0x8000
        for T in (n, 100, 33, 16, 1):
            G = eye[n - T:].contiguous()
            got = (q.qlora_fp8_linear_fwd(W, G, None, None, 0, 0.0) if ref is not wh else
                   q.qlora_fp8_linear_bwd(W, None, G, None, None, 0, 0.0)[0])
            assert np.array_equal(_no_minus_zero(host_bits(got)), _no_minus_zero(want[n - T:])), (n, T)


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_quantized_rows_keep_their_sign(T):
    """An identity weight shows the quantized rows, all 16 bits."""
    q = require_gpu()
    banner(f"fp8 signed identity T={T}")
    n = 320
    bits = synth.bf16_bits(synth.normal_f32(322, (T, n), 1.0))
    ref = synth.bf16_bits(ofp8.quantized_rows(odense.widen(bits)).astype(np.float32))
    W = q.qlora_fp8_quantize_weight(torch.eye(n, device="cuda"))
    Y = host_bits(q.qlora_fp8_linear_fwd(W, dev_bf16(bits), None, None, 0, 0.0))
    assert np.array_equal(_no_minus_zero(Y), _no_minus_zero(ref))
    dX = host_bits(q.qlora_fp8_linear_bwd(W, None, dev_bf16(bits), None, None, 0, 0.0)[0])
    assert np.array_equal(_no_minus_zero(dX), _no_minus_zero(ref))


def _bf16_parts(v, n):
    """v rounded to the sum of n bf16 parts."""
    total = np.zeros_like(v)
    for _ in range(n):
        total += onf4.bf16_bits_to_f32(synth.bf16_bits((v - total).astype(np.float32))).astype(np.float64)
    return total


@pytest.mark.parametrize("T,r", [(13, 16), (40, 8), (40, 32), (70, 48), (129, 64), (300, 65), (300, 128), (300, 200),
                                 (1000, 256)])
def test_adapter_gradients_are_held_to_32_bits(T, r):
    """One live token with three values, 1, 2^-8 and 2^-15, against factors of
    magnitude 1 to 2: U and V are sums a + b 2^-8 + c 2^-15 of bf16 numbers, 24
    bits from 2 down to 2^-22, exact in fp32, and need three bf16 parts.  dB's
    live rows are U, U 2^-8 and U 2^-15, dA's live columns the same of V, with s =
    1.  Three parts hold such a value; two leave up to 2^-16.  The bound is five
    additions (two for U, three for the parts) of at most one step of fp32
    each, 2^-23, should the matrix cores cut off instead of round."""
    q = require_gpu()
    banner(f"fp8 adapter gradients in 32 bits T={T} r={r}")
    n_in, n_out = 192, 320

    def factor(seed, shape):
        v = synth.normal_f32(seed, shape, 1.0)
        return synth.bf16_bits((np.sign(v) * (1 + np.floor(np.abs(v) * 1000) % 128 / 128)).astype(np.float32))
    A, B = factor(331, (r, n_in)), factor(332, (n_out, r))
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(333, (n_out, n_in), synth.W_STD)))
    t, steps = T // 2, (1.0, 2.0 ** -8, 2.0 ** -15)
    X = torch.zeros(T, n_in, dtype=torch.bfloat16, device="cuda")
    dY = torch.zeros(T, n_out, dtype=torch.bfloat16, device="cuda")
    kx, my = (5, 130, 70), (300, 64, 129)
    for s, k, m in zip(steps, kx, my):
        X[t, k], dY[t, m] = s, s
    Aw, Bw = odense.widen(A), odense.widen(B)
    U = sum(s * Aw[:, k] for s, k in zip(steps, kx))
    V = sum(s * Bw[m] for s, m in zip(steps, my))
    for v in (U, V):
        assert (v == v.astype(np.float32)).all() and (_bf16_parts(v, 3) == v).all()
        assert (np.abs(_bf16_parts(v, 2) - v) > 5 * 2.0 ** -23 * np.abs(v)).sum() >= r // 2  # two parts would not pass
    _, dA, dB = q.qlora_fp8_linear_bwd(W, X, dY, dev_bf16(A), dev_bf16(B), r, float(r))
    dA, dB = host(dA).astype(np.float64), host(dB).astype(np.float64)
    for s, k, m in zip(steps, kx, my):
        assert (np.abs(dA[:, k] - V * s) <= 5 * 2.0 ** -23 * np.abs(V * s)).all()
        assert (np.abs(dB[m] - U * s) <= 5 * 2.0 ** -23 * np.abs(U * s)).all()
    dA[:, list(kx)], dB[list(my)] = 0.0, 0.0
    assert not dA.any() and not dB.any()


# ------------------------------------------------------------------ workspaces, streams, graphs
@pytest.mark.parametrize("T,n_in,n_out,r", [
    (40, 2048, 2112, 16),     # K split both ways
    (5, 1024, 576, 24),       # U formed before the small forward
    (2, 1024, 4224, 8),       # the same for its many rows
    (9, 8256, 192, 8),        # few tokens by the GEMM's route
    (300, 4160, 1088, 64),    # K split in the forward alone
    (1500, 320, 256, 100),    # token slices of dA and dB
])
def test_workspace_contents_streams_and_graphs(T, n_in, n_out, r):
    q = require_gpu()
    banner(f"fp8 workspaces, streams, graphs T={T} {n_in}x{n_out} r={r}")
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(341, (n_out, n_in), synth.W_STD)))
    A, B = dev_bf16(_bf16(342, (r, n_in), 0.03)), dev_bf16(_bf16(343, (n_out, r), 0.05))
    X, dY = dev_bf16(_bf16(344, (T, n_in))), dev_bf16(_bf16(345, (T, n_out)))

    def both(ws=None):
        return (q.qlora_fp8_linear_fwd(W, X, A, B, r, 32.0, ws=ws),
                *q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, 32.0, ws=ws),
                q.qlora_fp8_linear_fwd(W, X, None, None, 0, 0.0, ws=ws),
                q.qlora_fp8_linear_bwd(W, None, dY, None, None, 0, 0.0, ws=ws)[0])

    def same(got, ref):
        return all(torch.equal(a, b) for a, b in zip(got, ref, strict=True))
    ref = [t.clone() for t in both()]
    assert all(bool(torch.isfinite(t).all()) for t in ref)
    need = max(q.qlora_fp8_workspace_bytes(T, n_in, n_out, rr, b) for rr in (0, r) for b in (False, True))
    for fill in (0x00, 0xff):
        assert same(both(torch.full((need,), fill, dtype=torch.uint8, device="cuda")), ref), fill
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert same(got, ref)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    keep, other = X.clone(), dev_bf16(_bf16(346, (T, n_in)))
    for turn in range(3):
        X.copy_(other if turn == 1 else keep)
        want = [t.clone() for t in both()]
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert same(out, want), turn


# ------------------------------------------------------------------ the largest sides
WIDEST = (1 << 24) - 64  # the other side 64: the expanded weight stays below 2^31 bytes


def _one_hot(T, n, at):
    x = torch.zeros(T, n, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(T, device="cuda"), at] = 1.0
    return x


@pytest.mark.parametrize("n_in,n_out", [(WIDEST, 64), (64, WIDEST)])
def test_widest_weights_are_read_exactly(n_in, n_out):
    """Offsets up to 2^31 within a tile, an output or a workspace: one value of 1 a
    row shows rows and columns of the weight, exactly."""
    q = require_gpu()
    banner(f"fp8 widest {n_in}x{n_out}")
    g = torch.Generator("cuda").manual_seed(351)
    W = q.qlora_fp8_quantize_weight(torch.randn(n_out, n_in, generator=g, device="cuda") * 0.02)
    wh = q.qlora_fp8_dequantize(W.codes, W.scales, n_out, n_in)
    for T in (1, 17, 33):
        for n, back in ((n_in, False), (n_out, True)):
            at = (torch.arange(T, device="cuda") * 2 + 1) * (n // (2 * T + 1))
            at[0], at[T - 1] = 0 if T > 1 else n - 1, n - 1
            X = _one_hot(T, n, at)
            if back:
                got, want = q.qlora_fp8_linear_bwd(W, None, X, None, None, 0, 0.0)[0], wh[at]
            else:
                got, want = q.qlora_fp8_linear_fwd(W, X, None, None, 0, 0.0), wh.t()[at]
            assert torch.equal(got, want), (T, back)  # (-0 equals 0)
            del X, got, want


@pytest.mark.parametrize("n_in,n_out", [((1 << 23) - 64, 64), (64, (1 << 23) - 64)])
@pytest.mark.parametrize("T", [3, 17])
def test_widest_adapters(T, n_in, n_out):
    """The adapter at the largest side it takes above 16 tokens.  X and dY have
    one value of 1 a row, so that U's and V's rows are columns of A and rows of B:
    Y and dX are sums of one weight and r products, dA and dB rows of V and U."""
    q = require_gpu()
    banner(f"fp8 widest adapter T={T} {n_in}x{n_out}")
    r, g = 8, torch.Generator("cuda").manual_seed(352)
    W = q.qlora_fp8_quantize_weight(torch.randn(n_out, n_in, generator=g, device="cuda") * 0.02)
    wh = q.qlora_fp8_dequantize(W.codes, W.scales, n_out, n_in)
    A = torch.randn(r, n_in, generator=g, device="cuda").to(torch.bfloat16)
    B = torch.randn(n_out, r, generator=g, device="cuda").to(torch.bfloat16)
    kx = torch.arange(T, device="cuda") * 3 % n_in if n_in == 64 else (n_in - 1 - torch.arange(T, device="cuda") * (n_in // T))
    my = torch.arange(T, device="cuda") * 3 % n_out if n_out == 64 else (n_out - 1 - torch.arange(T, device="cuda") * (n_out // T))
    assert len(set(kx.tolist())) == T and len(set(my.tolist())) == T
    X, dY = _one_hot(T, n_in, kx), _one_hot(T, n_out, my)
    Y = q.qlora_fp8_linear_fwd(W, X, A, B, r, float(r))
    dX, dA, dB = q.qlora_fp8_linear_bwd(W, X, dY, A, B, r, float(r))
    U, V = A.double().t()[kx], B.double()[my]

    def close(got, base, left, right):
        for t in range(T):  # a row at a time: the widest are 64 MiB in 64 bits
            terms = left[t][:, None] * right
            ref, mag = base[t].double() + terms.sum(0), base[t].double().abs() + terms.abs().sum(0)
            bound = 2.0 ** -8 * ref.abs() + 2.0 ** -12 * mag  # as in test_gpu_fp8.py
            assert bool(((got[t].double() - ref).abs() <= bound).all()), t
    close(Y, wh.t()[kx], U, B.double().t())
    close(dX, wh[my], V, A.double())
    # one term a sum, held to 32 bits: exact
    assert torch.equal(dA[:, kx], V.t().float()) and torch.equal(dB[my], U.float())
    dA[:, kx], dB[my] = 0.0, 0.0
    assert not bool(dA.any()) and not bool(dB.any())
