"""AdamW on the GPU: what an element that is not finite leaves alone, code for code, and
tensors of a plan against each of them alone.  Equalities bit for bit: an
element's result depends on its own values and, in 8 bits, on its block's largest and on
its place in the states."""

import numpy as np
import pytest
import torch

import synth

from gpu_util import banner, dev_f32, require_gpu

pytestmark = pytest.mark.gpu

RATES = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01)


@pytest.mark.parametrize("bits", [32, 8])
def test_blocks_of_states_that_are_not_finite(bits):
    """Each block's largest gradient is a known one, away from those that are not finite:
    scales and all other codes are the bits of the step without them, then and in
    the steps behind it."""
    q = require_gpu()
    banner(f"adamw blocks not finite {bits}")
    n, hit = 300, [5, 140, 299]
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[hit] = False
    runs = []
    for bad in (False, True):
        g = dev_f32(synth.normal_f32(6, (n,), 1.0)).clamp(-3, 3)
        g[[1, 131, 260]] = 50.0
        if bad:
            g[hit] = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda")
        p, f = torch.ones(n, dtype=torch.bfloat16, device="cuda"), torch.ones(n, device="cuda")
        state = q.qlora_adamw_state([n], bits, "cuda")
        plan = q.qlora_adamw_plan([p], [f], [g], state)
        seen = []
        for t in (1, 2, 3):
            q.qlora_adamw_step(plan, t, seed=9 + t, **RATES)
            seen.append([x.clone() for x in (p, f, state.m, state.v) + ((state.m_scales, state.v_scales) if bits == 8 else ())])
        runs.append(seen)
    for clean, dirty in zip(*runs):
        for k in range(4):
            assert torch.equal(dirty[k][:n][keep], clean[k][:n][keep]), k
            assert not dirty[k][n:].any()
        assert bool(torch.isnan(dirty[0][hit]).all()) and bool(torch.isnan(dirty[1][hit]).all())
        if bits == 8:
            assert torch.equal(dirty[4], clean[4]) and torch.equal(dirty[5], clean[5])
            assert bool(((dirty[2][hit] & 0x7f) == 0x7f).all()) and bool(((dirty[3][hit] & 0x7f) == 0x7f).all())
        else:
            assert not bool(torch.isfinite(dirty[2][hit]).any()) and not bool(torch.isfinite(dirty[3][hit]).any())


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_of_many_and_alone(bits):
    """1500 tensors in one plan, and some of them alone behind one that takes the place of
    all in front."""
    q = require_gpu()
    banner(f"adamw of many and alone {bits}")
    rng = np.random.Generator(np.random.PCG64(4))
    numels = [int(n) for n in rng.integers(0, 700, 1500)]
    numels[700:703] = [1, 2049, 8192]
    values = [rng.normal(0, 1, n).astype(np.float32) for n in numels]

    def step(sizes, grads):
        state = q.qlora_adamw_state(sizes, bits, "cuda")
        masters = [torch.ones(n, device="cuda") for n in sizes]
        plan = q.qlora_adamw_plan(None, masters, grads, state)
        for t in (1, 2):
            q.qlora_adamw_step(plan, t, seed=20 + t, **RATES)
        return masters, state, plan.offsets
    masters, state, offsets = step(numels, [dev_f32(v) for v in values])
    for i in (0, 1, 77, 700, 701, 702, 1499):
        n, o = numels[i], offsets[i]
        one, alone, where = step([o, n], [torch.full((o,), 0.5, device="cuda"), dev_f32(values[i])])
        assert where == [0, o] and torch.equal(one[1], masters[i])
        end = o + -(-n // 128) * 128
        assert torch.equal(alone.m[o:], state.m[o:end]) and torch.equal(alone.v[o:], state.v[o:end])
        if bits == 8:
            assert torch.equal(alone.m_scales[o // 128:], state.m_scales[o // 128:end // 128])
            assert torch.equal(alone.v_scales[o // 128:], state.v_scales[o // 128:end // 128])
