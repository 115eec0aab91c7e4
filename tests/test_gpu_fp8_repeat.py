"""The few-token forward of an 8-bit weight with rows of two chunks a wave and several
tiles a workgroup: every call gives the bits of the first, whatever ran in between, and
those are the oracle's to within the bounds of tests/test_gpu_fp8.py."""

import numpy as np
import pytest
import torch

import synth

from gpu_util import banner, dev_bf16, dev_f32, require_gpu
from test_gpu_fp8 import test_linear_matches_oracle as _matches_oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,n_in,n_out,r", [(2, 4160, 4224, 256), (1, 8192, 8256, 0), (16, 8192, 4160, 16), (3, 6208, 12352, 40)])
def test_every_call_gives_the_same_bits(T, n_in, n_out, r):
    q = require_gpu()
    banner(f"fp8 repeat T={T} {n_in}x{n_out} r={r}")
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(1, (n_out, n_in), synth.W_STD)))
    X = dev_bf16(synth.bf16_bits(synth.normal_f32(2, (T, n_in), 1.0)))
    A = dev_bf16(synth.bf16_bits(synth.normal_f32(3, (r, n_in), 0.05))) if r else None
    B = dev_bf16(synth.bf16_bits(synth.normal_f32(4, (n_out, r), 0.05))) if r else None
    first = q.qlora_fp8_linear_fwd(W, X, A, B, r, 16.0)
    flush = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for k in range(60):
        if k % 4 == 3:  # the weight comes from memory and not from the caches
            flush.fill_(k)
        differ += (q.qlora_fp8_linear_fwd(W, X, A, B, r, 16.0).view(torch.int16) != first.view(torch.int16)).sum()
    assert int(differ) == 0


def test_the_bits_are_right():
    _matches_oracle(2, 4160, 4224, 256, 16.0)
    _matches_oracle(3, 6208, 4160, 40, 80.0)
