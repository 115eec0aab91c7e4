"""A training step as it would be made: norm with 8-bit rows, an 8-bit layer with
an adapter, a norm, the output head's loss, the way back, the optimizer.  The
whole against the same steps in 64 bits with the layers' own quantizations."""

import numpy as np
import pytest
import torch

import synth
from oracle import adamw as oadamw
from oracle import dense as odense
from oracle import fp8 as ofp8
from oracle import head as ohead
from oracle import nf4 as onf4
from oracle import norm as onorm

from gpu_util import banner, dev_bf16, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _bf16(seed, shape, std=1.0):
    return synth.bf16_bits(synth.normal_f32(seed, shape, std))


def _wide(t):
    return onf4.bf16_bits_to_f32(host_bits(t)).astype(np.float64)


@pytest.mark.parametrize("T,bits", [(5, 32), (40, 8), (300, 32)])
def test_a_step(T, bits):
    """h = x + f(norm(x)) with f the 8-bit layer, logits = norm(h) W^T.  Each stage
    rounds to bf16 (1.7e-3 relative) or takes 8-bit codes of values that differ by that; ten
    such roundings, independent, are 5.4e-3: relative Frobenius 1e-2 for gradients, 1e-3
    for the loss, which is one number near log V."""
    q = require_gpu()
    banner(f"training step T={T} bits={bits}")
    H, V, r, alpha = 320, 704, 8, 16.0
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(1, (H, H), 0.05)))
    Wh = ofp8.dequantize(host(W.codes), host(W.scales))
    head = q.nf4_quantize_weight(dev_f32(synth.normal_f32(2, (V, H), 0.05)))
    Hv = _wide(q.nf4_dequantize(head.codes, head.absmax_q, head.absmax_scale, V * H)).reshape(V, H)
    A, B = dev_bf16(_bf16(3, (r, H), 0.05)), dev_bf16(_bf16(4, (H, r), 0.05))
    w1, w2 = dev_f32(1 + synth.normal_f32(5, (H,), 0.1)), dev_f32(1 + synth.normal_f32(6, (H,), 0.1))
    x = dev_bf16(_bf16(7, (T, H), 2.0))
    labels = np.random.Generator(np.random.PCG64(8)).integers(0, V, T)
    labels[::4] = -100
    y, g = torch.from_numpy(labels).cuda(), torch.full((T,), 1.0 / max(1, (labels >= 0).sum()), device="cuda")
    dA, dB, dw1, dw2 = torch.empty(r, H, device="cuda"), torch.empty(H, r, device="cuda"), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    master = [A.float(), B.float(), w1, w2]
    start = [t.clone() for t in master]
    state = q.qlora_adamw_state([t.numel() for t in master], bits, "cuda")
    plan = q.qlora_adamw_plan([A, B, None, None], master, [dA, dB, dw1, dw2], state)

    def step(t):
        n1, rows, _, s1 = q.qlora_rmsnorm_fwd(x, w1, eps=EPS, rows8=True)
        f = q.qlora_fp8_linear_fwd_rows(W, rows, n1, A, B, r, alpha)
        n2, _, h, s2 = q.qlora_rmsnorm_fwd(f, w2, residual=x, eps=EPS)
        loss, _, dn2 = q.qlora_head_loss_grad(head, n2, y, g)
        dh, _ = q.qlora_rmsnorm_bwd(dn2, h, w2, s2, dweight=dw2)
        dn1, _, _ = q.qlora_fp8_linear_bwd(W, n1, dh, A, B, r, alpha, dA=dA, dB=dB)
        dx, _ = q.qlora_rmsnorm_bwd(dn1, x, w1, s1, dres=dh, dweight=dw1)
        q.qlora_adamw_step(plan, t, lr=1e-2, weight_decay=0.1)
        return loss, dx

    A0, B0, v1, v2 = _wide(A), _wide(B), host(w1).astype(np.float64), host(w2).astype(np.float64)
    loss, dx = step(1)
    torch.cuda.synchronize()
    X, s = _wide(x), alpha / r
    m1, o1 = onorm.fwd(X, v1, EPS)
    hh = X + ofp8.quantized_rows(m1) @ Wh.T + s * (m1 @ A0.T) @ B0.T
    m2, o2 = onorm.fwd(hh, v2, EPS)
    rl, _, dm2, _, _ = ohead.loss_grad(m2, Hv, labels, host(g).astype(np.float64))
    dhh, rw2, _, _ = onorm.bwd(dm2, hh, v2, o2)
    dm1, rA, rB = ofp8.linear_bwd(Wh, m1, dhh, A0, B0, r, alpha)
    rx, rw1, _, _ = onorm.bwd(dm1, X, v1, o1, dhh)
    got = {"loss": host(loss), "dx": _wide(dx), "dA": host(dA), "dB": host(dB), "dw1": host(dw1), "dw2": host(dw2)}
    ref = {"loss": rl, "dx": rx, "dA": rA, "dB": rB, "dw1": rw1, "dw2": rw2}
    off = {k: odense.rel_frobenius(got[k], ref[k]) for k in got}
    print(off, flush=True)
    # the 8-bit codes of dh differ where its own error crosses a border of codes: half a code step
    # (2^-4) at the share of values whose 1.7e-3 error crosses one, 2^-4 sqrt(2 * 1.7e-3 / 2^-3) = 1.0e-2 of dX's first part
    assert off.pop("dx") <= 1.5e-2 and off.pop("dw1") <= 2e-2 and off.pop("loss") <= 1e-3
    assert max(off.values()) <= 1e-2, off
    # the optimizer on the gradients that the step left
    for p, b, d in zip(master, start, (dA, dB, dw1, dw2)):
        want, _, _ = oadamw.step(host(b).astype(np.float64), host(d).astype(np.float64), 0.0, 0.0, 1, 1e-2, .9, .999, 1e-8, .1)
        assert np.abs(host(p) - want).max() <= 1e-6
    assert torch.equal(A, master[0].to(torch.bfloat16)) and torch.equal(B, master[1].to(torch.bfloat16))

    # the whole step in a graph, next to eager steps: the same bits from the same state
    keep = [*master, A, B, state.m, state.v] + ([state.m_scales, state.v_scales] if bits == 8 else [])
    now = [t.clone() for t in keep]
    outs = [t.clone() for t in step(2)]
    after = [t.clone() for t in keep]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(2)
    for turn in range(3):
        for t, c in zip(keep, now):
            t.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, outs)), turn
        assert all(torch.equal(a, b) for a, b in zip(keep, after)), turn
        for t, c in zip(keep, now):
            t.copy_(c)
        again = step(2)
        assert all(torch.equal(a, b) for a, b in zip(again, outs))
