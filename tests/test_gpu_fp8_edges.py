"""The 8-bit linear layer where its inputs leave the ordinary: rows that are
not finite, adapter products past bf16's largest, in the forward and in the
gradients."""

import numpy as np
import pytest
import torch

import synth
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
