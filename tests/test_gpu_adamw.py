"""The AdamW step on the GPU against oracle/adamw.py in 64 bits.

Tolerances, u = 2^-24 (fp32's half step).  m and v: two products and a sum, with a
gradient that may carry one more rounding (v: two): 4 u (|b1 m| + |c1 g|) and 5 u v;
the constants, rounded to fp32, add u each.  The update: m within 5 u, sqrt v within 4 u, two more
products, a sum, a quotient, the rate: 16 u of lr / (1 - b1^t) |m| / (...) and, where m cancels, its absolute
error through the same factor; decay and the two differences: 4 u (|p| + update).  A bf16
parameter: 2^-8 of the value on top.

8 bits: scales and codes have to be the oracle's, except where the value before the
rounding down lies within its own error of a whole number of steps: r = sqrt v and m are
within 8 u of the value (m: of its terms), so the number of steps is off by at most
16 * 8 u = 2^-17 of the terms' sum over the value; there a code may be the next one."""

import numpy as np
import pytest
import torch

import synth
from oracle import adamw as oadamw
from oracle import fp8 as ofp8
from oracle import nf4 as onf4

from gpu_util import banner, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RATES = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def _wide(t):
    return (onf4.bf16_bits_to_f32(host_bits(t)) if t.dtype == torch.bfloat16 else host(t)).astype(np.float64).reshape(-1)


# numels: one, next to a lane's eight, a block's 128, a chunk's 2048; none; larger than several chunks
SETS = [[1], [7, 8, 9], [127, 128, 129], [2047, 2048, 2049], [0, 5, 0, 130, 0], [16 * 4096, 4096 * 16, 333, 10001]]
FORMS = ["both", "master", "param", "mixed"]


def _make(q, numels, bits, form, seed, guard=64):
    """Tensors in the middle of larger ones whose rest is a mark; states that a run
    would have."""
    rng = np.random.Generator(np.random.PCG64(seed))
    params, masters, grads, around = [], [], [], []

    def inside(values, dtype, mark):
        n = len(values)
        big = torch.full((guard + n + guard,), mark, dtype=dtype, device="cuda")
        big[guard:guard + n] = torch.from_numpy(values).to(dtype).cuda()
        around.append((big, guard, n, mark))
        return big[guard:guard + n]
    for i, n in enumerate(numels):
        kind = form if form != "mixed" else ("both", "master", "param")[i % 3]
        size = 10.0 ** rng.uniform(-4, 0)
        w = rng.normal(0, 0.05, n).astype(np.float32)
        masters.append(inside(w, torch.float32, 3.0) if kind != "param" else None)
        params.append(inside(w, torch.bfloat16, 3.0) if kind != "master" else None)
        grads.append(inside((rng.normal(0, size, n) * np.exp(rng.normal(0, 1, n))).astype(np.float32), torch.float32, 3.0))
    length = q.qlora_adamw_state_len(numels)
    m, r = np.zeros(length), np.zeros(length)
    at = 0
    for n, g in zip(numels, grads):
        gs = np.abs(_wide(g))
        m[at:at + n] = 0.3 * gs * rng.normal(0, 1, n)
        r[at:at + n] = gs * rng.uniform(0.3, 2, n)
        if n > 20:
            m[at + 3], r[at + 3] = 0, 0
            r[at + 5] *= 1e-7
        at += -(-n // 128) * 128
    if bits == 32:
        state = q.AdamWState(dev_f32(m), dev_f32(r * r))
    else:
        parts = []
        for x in (m, r):
            e = ofp8.scale_exponent(np.abs(x.reshape(-1, 128)).max(axis=1))
            parts.append((ofp8.encode((x.reshape(-1, 128) / np.exp2(e.astype(np.float64))[:, None])).reshape(-1), (e + 127).astype(np.uint8)))
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        state = q.AdamWState(t(parts[0][0]), t(parts[1][0]), t(parts[0][1]), t(parts[1][1]))
    return params, masters, grads, state, around


def _values(state, bits):
    """(m, v) of a state in 64 bits."""
    if bits == 32:
        return _wide(state.m), _wide(state.v)
    m = oadamw.from8(host(state.m), host(state.m_scales))
    r = oadamw.from8(host(state.v), host(state.v_scales))
    return m, r * r


def _check_codes(codes, scales, x, terms, u, keep):
    """One tensor's codes and scales against the values x; terms: the size of what x
    was added up from."""
    n = len(x)
    val, sc, y, d = oadamw.to8(x, u, keep)
    got = ofp8.e4m3_values()[codes[:n]]
    f = np.repeat(np.exp2(scales.astype(np.float64) - 127), 128)[:n]
    if not np.array_equal(scales, sc):  # a largest value next to 448 2^e
        for b in np.flatnonzero(scales != sc):
            top = np.abs(x[b * 128:b * 128 + 128]).max()
            assert abs(int(scales[b]) - int(sc[b])) == 1
            assert abs(top / (448 * 2.0 ** (min(scales[b], sc[b]) - 127.0)) - 1) <= 2.0 ** -19
    same = np.repeat(scales == sc, 128)[:n]
    steps = np.abs(y) / d + u[:n]
    near = np.abs(steps - np.rint(steps)) <= 2.0 ** -17 * np.maximum(terms / np.maximum(np.abs(x), 1e-300), 1)
    diff = got != val
    assert not (diff & same & ~near).any(), np.flatnonzero(diff & same & ~near)[:5]
    assert (np.abs(got - val)[diff & same] <= d[diff & same] * (1 + 1e-9)).all()
    # however the noise falls, a code is within a step of its value
    assert (np.abs(got * f - x) <= 2.0 ** -2 * np.abs(x) + f * 2.0 ** -8).all()
    assert not codes[n:].any()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("numels", SETS, ids=lambda s: "_".join(map(str, s)))
def test_steps(bits, form, numels):
    q = require_gpu()
    banner(f"adamw {bits} {form} {numels}")
    params, masters, grads, state, around = _make(q, numels, bits, form, 7 + len(numels))
    plan = q.qlora_adamw_plan(params, masters, grads, state)
    assert plan.bits == bits
    for t, clip in ((1, None), (50, 0.37)):
        scale = None if clip is None else torch.tensor([clip], device="cuda")
        s = 1.0 if clip is None else float(np.float32(clip))
        m0, v0 = _values(state, bits)
        before = [_wide(f if f is not None else p) for p, f in zip(params, masters)]
        seed = 1000 + t
        q.qlora_adamw_step(plan, t, grad_scale=scale, seed=seed, **RATES)
        m1, v1 = (_wide(state.m), _wide(state.v)) if bits == 32 else (None, None)
        um, ur = oadamw.noise(len(m0), seed)
        for i, n in enumerate(numels):
            o = plan.offsets[i]
            g = _wide(grads[i]) * s
            rp, rm, rv = oadamw.step(before[i], g, m0[o:o + n], v0[o:o + n], t, RATES["lr"], RATES["beta1"], RATES["beta2"],
                                     RATES["eps"], RATES["weight_decay"])
            terms = RATES["beta1"] * np.abs(m0[o:o + n]) + (1 - RATES["beta1"]) * np.abs(g)
            if bits == 32:
                assert (np.abs(m1[o:o + n] - rm) <= 5 * U * terms + 1e-44).all()
                assert (np.abs(v1[o:o + n] - rv) <= 6 * U * rv + 1e-44).all()
                end = -(-n // 128) * 128
                assert not m1[o + n:o + end].any() and not v1[o + n:o + end].any()
            elif n:
                end = -(-n // 128) * 128
                _check_codes(host(state.m)[o:o + end], host(state.m_scales)[o // 128:(o + end) // 128], rm, terms, um[o:o + end], False)
                _check_codes(host(state.v)[o:o + end], host(state.v_scales)[o // 128:(o + end) // 128], np.sqrt(rv), np.sqrt(rv), ur[o:o + end], True)
                sign = (host(state.m)[o:o + n] & 0x80) != 0
                assert np.array_equal(sign[rm != 0], rm[rm != 0] < 0)
            factor = RATES["lr"] / (1 - RATES["beta1"] ** t) / (np.sqrt(rv / (1 - RATES["beta2"] ** t)) + RATES["eps"])
            moved = factor * np.abs(rm)
            bound = 16 * U * moved + factor * 5 * U * terms + 4 * U * (np.abs(before[i]) + moved) + 1e-44
            if masters[i] is not None:
                assert (np.abs(_wide(masters[i]) - rp) <= bound).all()
                if params[i] is not None:
                    assert torch.equal(params[i], masters[i].to(torch.bfloat16))
            else:
                assert (np.abs(_wide(params[i]) - rp) <= bound + 2.0 ** -8 * (np.abs(rp) + bound)).all()
    for big, a, n, mark in around:  # nothing beside the tensors is written
        assert bool((big[:a] == mark).all()) and bool((big[a + n:] == mark).all())


def test_zero_states_and_gradients():
    """From nothing: a zero gradient leaves zero states and decays the parameter
    alone, a first gradient moves it by lr."""
    q = require_gpu()
    banner("adamw from zero")
    for bits in (32, 8):
        p, g = torch.ones(300, device="cuda"), torch.zeros(300, device="cuda")
        state = q.qlora_adamw_state([300], bits, "cuda")
        plan = q.qlora_adamw_plan(None, [p], [g], state)
        q.qlora_adamw_step(plan, 1, lr=0.5, weight_decay=0.5)
        assert bool((p == 0.75).all()) and not state.m.any() and not state.v.any()
        g[7] = -1e-3
        q.qlora_adamw_step(plan, 1, lr=0.5)
        assert abs(p[7].item() - 1.25) < 1e-5 and bool((p[:7] == 0.75).all())


def test_a_small_second_moment_does_not_vanish():
    """An element whose sqrt v is 2^-40 of its block's largest keeps the smallest
    code, so that its momentum is not divided by eps alone.  With m at the smallest code too, the
    next step with no gradient moves it by at most lr m / sqrt v."""
    q = require_gpu()
    banner("adamw small v")
    p, g = torch.zeros(128, device="cuda"), torch.zeros(128, device="cuda")
    g[0], g[1] = 1.0, 2.0 ** -40
    state = q.qlora_adamw_state([128], 8, "cuda")
    plan = q.qlora_adamw_plan(None, [p], [g], state)
    q.qlora_adamw_step(plan, 1, lr=1e-3, seed=3)
    codes = host(state.v)
    assert codes[1] == 1 and not codes[2:].any()
    g.zero_()
    before = p.clone()
    for t in range(2, 12):
        q.qlora_adamw_step(plan, t, lr=1e-3, seed=t)
    moved = (p - before).abs()
    assert host(state.v)[1] >= 1 and not moved[2:].any()
    # smallest codes: m 2^-9 448^-1 0.1, sqrt v 2^-9 448^-1 0.0316 of the largest's: ratio 3.2 a step at most, corrected
    assert moved[1].item() <= 10 * 1e-3 * 4


def test_mean_over_seeds_is_the_value():
    """The 8-bit states of 400 seeds average to the 32-bit ones: a code's noise is
    uniform over a step (its standard deviation at most half a step), so the mean of 400 is within 5 half
    steps / 20; step <= 2^-3 of the value or 2^-9 of the scale."""
    q = require_gpu()
    banner("adamw mean over seeds")
    n = 256
    g = dev_f32(synth.normal_f32(5, (n,), 1.0))
    p = torch.zeros(n, device="cuda")
    exact = q.qlora_adamw_state([n], 32, "cuda")
    q.qlora_adamw_step(q.qlora_adamw_plan(None, [p], [g], exact), 1, lr=0.0)
    sm, sr = np.zeros(n), np.zeros(n)
    for seed in range(400):
        state = q.qlora_adamw_state([n], 8, "cuda")
        q.qlora_adamw_step(q.qlora_adamw_plan(None, [p], [g], state), 1, lr=0.0, seed=seed)
        sm += oadamw.from8(host(state.m), host(state.m_scales))
        sr += oadamw.from8(host(state.v), host(state.v_scales))
    for got, x in ((sm / 400, _wide(exact.m)), (sr / 400, np.sqrt(_wide(exact.v)))):
        top = np.repeat(np.abs(x.reshape(-1, 128)).max(axis=1), 128)
        step = np.maximum(2.0 ** -3 * np.abs(x), 2.0 ** -16 * top)
        assert (np.abs(got - x) <= 5 * step / 40 + step / 512).all()


def test_states_that_are_not_finite_stay_alone():
    q = require_gpu()
    banner("adamw not finite")
    for bits in (32, 8):
        out = []
        for bad in (False, True):
            g = dev_f32(synth.normal_f32(6, (300,), 1.0))
            if bad:
                g[5], g[140], g[299] = float("nan"), float("inf"), float("-inf")
            p = torch.ones(300, dtype=torch.bfloat16, device="cuda")
            state = q.qlora_adamw_state([300], bits, "cuda")
            q.qlora_adamw_step(q.qlora_adamw_plan([p], None, [g], state), 1, lr=1e-2, seed=9)
            out.append((p, state))
        (p0, s0), (p1, s1) = out
        hit = torch.zeros(300, dtype=torch.bool, device="cuda")
        hit[[5, 140, 299]] = True
        assert bool(torch.isnan(p1[hit]).all()) and torch.equal(p1[~hit], p0[~hit])
        if bits == 8:
            assert bool(((s1.m[:300][hit] & 0x7f) == 0x7f).all()) and bool(((s1.v[:300][hit] & 0x7f) == 0x7f).all())
            # the largest of each block was another element: the rest is as it was
            if torch.equal(s0.m_scales, s1.m_scales):
                assert torch.equal(s1.m[:300][~hit], s0.m[:300][~hit])
        else:
            assert not bool(torch.isfinite(s1.v[:300][hit]).any()) and torch.equal(s1.v[:300][~hit], s0.v[:300][~hit])


def test_many_tensors_streams_graphs_and_plans():
    """More tensors than one launch of the plan takes, of many sizes; the step is
    the same bits on another stream, in graphs, and for each tensor alone where
    its states start at the same place."""
    q = require_gpu()
    banner("adamw many tensors")
    rng = np.random.Generator(np.random.PCG64(3))
    numels = [int(n) for n in rng.integers(0, 700, 180)] + [50000]
    for bits in (32, 8):
        def fresh():
            params, masters, grads, state, _ = _make(q, numels, bits, "mixed", 11)
            return params, masters, grads, state

        def result(params, masters, state):
            ts = [t for t in params + masters + [state.m, state.v, state.m_scales, state.v_scales] if t is not None]
            return [t.clone() for t in ts]

        def two(plan):
            q.qlora_adamw_step(plan, 3, seed=5, **RATES)
            q.qlora_adamw_step(plan, 4, seed=6, **RATES)
        a = fresh()
        two(q.qlora_adamw_plan(*a[:3], a[3]))
        ref = result(a[0], a[1], a[3])
        a = fresh()
        side = torch.cuda.Stream()
        # (the plan waits for the current stream: the side stream finds it whole)
        plan = q.qlora_adamw_plan(*a[:3], a[3])
        with torch.cuda.stream(side):
            two(plan)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(result(a[0], a[1], a[3]), ref))
        # captured steps, replayed on restored values
        a = fresh()
        start = result(a[0], a[1], a[3])
        keep = [t for t in a[0] + a[1] + [a[3].m, a[3].v, a[3].m_scales, a[3].v_scales] if t is not None]
        plan = q.qlora_adamw_plan(*a[:3], a[3])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            with pytest.raises(RuntimeError, match="captured"):
                q.qlora_adamw_plan(*a[:3], a[3])
            two(plan)
        for turn in range(3):
            for t, s in zip(keep, start):
                t.copy_(s)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(result(a[0], a[1], a[3]), ref)), turn


def test_plan_keeps_its_tensors():
    q = require_gpu()
    banner("adamw plan keeps tensors")
    state = q.qlora_adamw_state([4096], 32, "cuda")
    p, g = torch.zeros(4096, device="cuda"), torch.ones(4096, device="cuda")
    plan = q.qlora_adamw_plan(None, [p], [g], state)
    alias = plan.tensors[0]
    del p, g, state
    torch.cuda.empty_cache()
    other = [torch.full((4096,), 9.0, device="cuda") for _ in range(8)]
    q.qlora_adamw_step(plan, 1, lr=0.5)
    torch.cuda.synchronize()
    assert all(bool((t == 9).all()) for t in other) and bool(((alias + 0.5).abs() < 1e-4).all())


def test_table_outlives_a_step_on_another_stream():
    q = require_gpu()
    banner("adamw table on another stream")
    state = q.qlora_adamw_state([3 << 20], 32, "cuda")
    p, g = torch.zeros(3 << 20, device="cuda"), torch.ones(3 << 20, device="cuda")
    plan = q.qlora_adamw_plan(None, [p], [g], state)
    at, size = plan.table.data_ptr(), plan.table.numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        q.qlora_adamw_step(plan, 1, lr=0.5)
    del plan
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query() and all(t.data_ptr() != at for t in others)
    torch.cuda.synchronize()
    assert bool(((p + 0.5).abs() < 1e-4).all())


def test_refusals():
    q = require_gpu()
    banner("adamw refusals")
    p, f, g = torch.zeros(40, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(40, 8, device="cuda"), torch.zeros(40, 8, device="cuda")
    state = q.qlora_adamw_state([320], 8, "cuda")
    ok = q.qlora_adamw_plan([p], [f], [g], state)

    def refused(error, *args):
        with pytest.raises(error):
            q.qlora_adamw_plan(*args)
    refused(TypeError, [None], [None], [g], state)
    refused(TypeError, [p.float()], None, [g], state)
    refused(TypeError, [p], None, [g.double()], state)
    refused(TypeError, [p], None, [None], state)
    refused(ValueError, [p.t()], None, [g.t()], state)
    refused(ValueError, [p[:20]], None, [g], state)
    refused(ValueError, [p.view(8, 40)], None, [g], state)
    refused(ValueError, [p.cpu()], None, [g], state)
    refused(ValueError, [p, p], None, [g], state)
    refused(ValueError, [p], None, [g], q.qlora_adamw_state([400], 8, "cuda"))
    refused(TypeError, [p], None, [g], q.AdamWState(state.m, state.v.float(), state.m_scales, state.v_scales))
    refused(q.QloraError, [p, p], None, [g, g], q.qlora_adamw_state([320, 320], 8, "cuda"))
    refused(q.QloraError, None, [f], [f], state)
    for kw in ({"lr": float("nan")}, {"lr": 1e-3, "beta1": 1.0}, {"lr": 1e-3, "eps": -1.0}):
        with pytest.raises(q.QloraError):
            q.qlora_adamw_step(ok, 1, **kw)
    with pytest.raises(q.QloraError):
        q.qlora_adamw_step(ok, 0, lr=1e-3)
    with pytest.raises(ValueError):
        q.qlora_adamw_step(ok, 1, lr=1e-3, grad_scale=torch.ones(1))
    twice = q.AdamWState(state.m, state.m, state.m_scales, state.v_scales)
    with pytest.raises(q.QloraError):
        q.qlora_adamw_step(q.qlora_adamw_plan([p], [f], [g], twice), 1, lr=1e-3)
    with pytest.raises(ValueError):
        q.qlora_adamw_state([5], 16, "cuda")
