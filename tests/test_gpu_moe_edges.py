"""The mixture-of-experts operators where their inputs leave the ordinary:
NaN and infinities in rows and in masked places, hidden values past bf16's
largest, workspaces with any contents."""

import numpy as np
import pytest
import torch

import synth
from oracle import moe as omoe
from oracle import nf4 as onf4

import test_gpu_moe
from gpu_util import banner, dev_bf16, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu

# a sum of at most 1024 terms, an exponential and a handful of products, as in test_gpu_moe.py
FP32 = 64 * 2.0 ** -24


def _grad(q, l, ids, dw, renorm):
    return host(q.qlora_moe_route_bwd(dev_f32(l), torch.from_numpy(ids).cuda(), dev_f32(dw), renormalize=renorm))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [4, 12, 60, 128, 200, 1000])
def test_route_gradient_of_a_nan_row_is_nan(E, renorm):
    """Every logit the weights were taken from is NaN (as after a token whose
    hidden state is NaN), or some are: the weights are NaN and so is the
    gradient.  A row of nothing but -inf beside them keeps its zeros."""
    q = require_gpu()
    banner(f"route gradient of NaN rows E={E} renorm={renorm}")
    k = 4
    l = synth.normal_f32(201, (6, E), 1.0)
    l[1] = np.nan
    l[2, 0] = np.nan
    l[3] = -np.inf
    l[4] = -np.inf
    l[4, E - 1] = np.nan                         # the only one that is not masked
    dw = synth.normal_f32(202, (6, k), 1.0)
    ids, w = q.qlora_moe_route(dev_f32(l), k, renormalize=renorm)
    ids, w = host(ids), host(w)
    assert np.isnan(w[[1, 2, 4]]).all() and not w[3].any()
    dl = _grad(q, l, ids, dw, renorm)
    for t in (1, 2, 4):
        chosen = np.isin(np.arange(E), ids[t]) if renorm else np.ones(E, bool)
        assert np.isnan(dl[t, chosen]).all(), t
    assert not dl[3].any()
    fine = [0, 5]
    assert np.abs(dl[fine] - omoe.route_bwd(l[fine], ids[fine], dw[fine], renorm)).max() <= FP32 * 2 * np.abs(dw).max()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("E", [6, 60, 200])
def test_route_gradient_of_masked_choices_counts_for_nothing(E, bad, renorm):
    """A choice whose logit is -inf (fewer than k experts were left, or the row
    is padding) has weight 0, whatever the logits: what stands in its place of
    dweights, an infinity or a NaN, changes nothing.  The other rows are the
    ones of finite gradients."""
    q = require_gpu()
    banner(f"route gradient of masked choices E={E} {bad} renorm={renorm}")
    k = 4
    l = synth.normal_f32(203, (5, E), 1.0)
    l[1] = -np.inf                               # no choice at all
    l[2, 1:] = -np.inf                           # one
    l[3, 3:] = -np.inf                           # three
    dw = synth.normal_f32(204, (5, k), 1.0)
    clean = dw.copy()
    dw[1], dw[2, 1:], dw[3, 3] = bad, bad, bad
    clean[1], clean[2, 1:], clean[3, 3] = 0.0, 0.0, 0.0
    ids, w = q.qlora_moe_route(dev_f32(l), k, renormalize=renorm)
    ids = host(ids)
    assert not host(w)[1].any() and not host(w)[2, 1:].any() and host(w)[3, 3] == 0
    dl = _grad(q, l, ids, dw, renorm)
    assert not dl[1].any()
    assert np.array_equal(dl, _grad(q, l, ids, clean, renorm))
    assert np.abs(dl - omoe.route_bwd(l, ids, clean, renorm)).max() <= FP32 * 2 * np.abs(clean).max()


@pytest.mark.parametrize("T,E,k,H,I", [
    (4, 2, 1, 64, 64),        # the down product in one launch
    (40, 2, 2, 64, 128),      # in two, two column tiles at a time
    (5, 60, 4, 256, 1024),    # one
    (64, 60, 8, 128, 512),    # more than 64 pairs
])
def test_experts_hidden_values_past_bf16(T, E, k, H, I):
    """Hidden values are kept as bf16 pairs hi + lo.  One between bf16's largest
    and fp32's has to stay the finite number it is, an infinite one infinite
    with its sign: the lo of an infinite hi must not be inf - inf.

    All weights of the gate and up products are c = 181/128 (its block's
    absmax and its group's: exact in the 4-bit format), all of the down
    product 2^-10.  x has one value, 181/128 2^63: g = u = 1.99957 2^63, exact, h
    = 1.99915 2^127, above bf16's largest (1.99219 2^127) by more than the half
    step that still rounds to it; silu(g) = g, since exp(-g) is 0."""
    q = require_gpu()
    banner(f"moe hidden values past bf16 T={T} E={E} k={k} H={H} I={I}")
    c, d = 181 / 128, 2.0 ** -10
    gu = q.nf4_quantize_weight(torch.full((E * 2 * I, H), c, device="cuda"))
    dn = q.nf4_quantize_weight(torch.full((E * H, I), d, device="cuda"))
    x = np.zeros((T, H), dtype=np.float64)
    x[0, H // 2] = c * 2.0 ** 63                 # h in (bf16's largest, fp32's largest)
    x[1, 3] = 2.0 ** 100                         # h infinite
    x[2:] = synth.normal_f32(205, (T - 2, H), 1.0)
    x[3] = 0.0
    bits = synth.bf16_bits(x.astype(np.float32))
    x = onf4.bf16_bits_to_f32(bits).astype(np.float64)
    ids = np.tile(np.arange(k, dtype=np.int32), (T, 1))
    w = np.abs(synth.normal_f32(206, (T, k), 0.25)) + 0.125
    w /= 16 * k                                  # Y of row 0 stays finite
    sign = np.ones(T, np.float32)
    sign[1] = -1.0
    w = (w * sign[:, None]).astype(np.float32)
    Y = onf4.bf16_bits_to_f32(host_bits(q.qlora_moe_fwd(gu, dn, E, dev_bf16(bits), torch.from_numpy(ids).cuda(),
                                                        dev_f32(w)))).astype(np.float64)
    g = c * x.sum(1)                             # the same in every gate, up and down row
    with np.errstate(over="ignore"):
        h = g / (1 + np.exp(-g)) * g
    assert (2 - 2.0 ** -8) * 2.0 ** 127 < h[0] < np.finfo(np.float32).max < h[1]
    ref = w.astype(np.float64).sum(1) * I * d * h
    assert np.isneginf(Y[1]).all()
    fine = np.arange(T) != 1
    # row 0 and the others: the final rounding, 2^-8, and 2^-13 of the terms' magnitudes
    # as for any row; x of the others adds up H terms of both signs in fp32, at most
    # H 2^-24 of their magnitudes, twice, in g and u
    mag = np.abs(w).sum(1) * I * d * np.abs(h)
    drift = np.abs(w).sum(1) * I * d * 4 * np.abs(g) * c * np.abs(x).sum(1) * H * 2.0 ** -24
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * mag + drift + 1e-37
    assert (np.abs(Y - ref[:, None]) <= bound[:, None])[fine].all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [8, 60, 300])
def test_route_gradient_of_zeros_is_zero(E, renorm):
    q = require_gpu()
    banner(f"route gradient of zeros E={E} renorm={renorm}")
    l = synth.normal_f32(207, (9, E), 3.0)
    l[4] = -np.inf
    l[5, 2:] = -np.inf
    ids, _ = q.qlora_moe_route(dev_f32(l), 4, renormalize=renorm)
    assert not _grad(q, l, host(ids), np.zeros((9, 4), np.float32), renorm).any()


@pytest.mark.parametrize("T,E,k,H,I", [
    (5, 8, 2, 256, 320),      # at most 64 pairs, the down product in one launch
    (9, 8, 4, 448, 1024),     # in two launches
    (40, 60, 4, 320, 192),    # more than 64 pairs
    (64, 4, 8, 256, 320),     # two column tiles at a time, more of them than one
    (61, 4, 4, 576, 256),     # column tiles shared by several workgroups
])
def test_experts_workspace_contents(T, E, k, H, I):
    """The pairs that are no choice leave their part of the workspace unwritten:
    whatever it holds, the result is the same bit for bit, and a row of nothing
    but such pairs is 0."""
    q = require_gpu()
    banner(f"moe workspace contents T={T} E={E} k={k} H={H} I={I}")
    gu = q.nf4_quantize_weight(dev_f32(synth.normal_f32(208, (E * 2 * I, H), H ** -0.5)))
    dn = q.nf4_quantize_weight(dev_f32(synth.normal_f32(209, (E * H, I), I ** -0.5)))
    rng = np.random.Generator(np.random.PCG64(T * E))
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.3] = -1
    ids[0] = [E, -1, -7, 1 << 30][:k] + [-1] * (k - 4)
    ids[T - 1] = -1
    ids, X = torch.from_numpy(ids).cuda(), dev_bf16(synth.bf16_bits(synth.normal_f32(210, (T, H), 1.0)))
    w = dev_f32(synth.normal_f32(211, (T, k), 1.0))
    need = q.qlora_moe_workspace_bytes(T, H, I, k)
    Y = q.qlora_moe_fwd(gu, dn, E, X, ids, w)
    assert bool(torch.isfinite(Y).all()) and not Y[[0, T - 1]].any() and bool(Y[1:T - 1].any())
    for fill in (0x00, 0x7f, 0xff):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(q.qlora_moe_fwd(gu, dn, E, X, ids, w, ws=ws), Y), fill


@pytest.mark.parametrize("T,E,k,H,I", [(64, 600, 8, 128, 128), (20, 1024, 16, 128, 256), (13, 80, 6, 128, 128)])
def test_more_experts_than_pairs(T, E, k, H, I):
    """More than 64 pairs over even more experts: a workgroup's slot is a pair,
    and only an expert's first pair works."""
    test_gpu_moe.test_experts_where_the_kernels_change(T, E, k, H, I)


@pytest.mark.parametrize("T,k,H,I", [(1, 1, (1 << 20) - 64, 64), (17, 2, (1 << 20) - 64, 64), (17, 2, 64, (1 << 20) - 64),
                                     (64, 3, (1 << 20) - 64, 128)])
def test_experts_widest_sides(T, k, H, I):
    """hidden and inter next to their limit of 2^20."""
    q = require_gpu()
    banner(f"moe widest T={T} k={k} H={H} I={I}")
    E, g = 3, torch.Generator("cuda").manual_seed(221)
    gu = q.nf4_quantize_weight(torch.randn(E * 2 * I, H, generator=g, device="cuda") * H ** -0.5)
    dn = q.nf4_quantize_weight(torch.randn(E * H, I, generator=g, device="cuda") * I ** -0.5)
    X = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).to(torch.int32)
    w = torch.randn(T, k, generator=g, device="cuda")
    Y = q.qlora_moe_fwd(gu, dn, E, X, ids, w)

    vg = q.nf4_dequantize(gu.codes, gu.absmax_q, gu.absmax_scale, E * 2 * I * H).view(E, 2 * I, H)
    vd = q.nf4_dequantize(dn.codes, dn.absmax_q, dn.absmax_scale, E * H * I).view(E, H, I)
    ref, mag = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        took = (w.double() * (ids == e)).sum(1)
        rows = (ids == e).any(1).nonzero().view(-1)
        if not rows.numel():
            continue
        gate = X[rows].double() @ vg[e].double().t().contiguous()
        h = gate[:, :I] * torch.sigmoid(gate[:, :I]) * gate[:, I:]
        down = vd[e].double().t().contiguous()
        ref[rows] += took[rows, None] * (h @ down)
        mag[rows] += took[rows, None].abs() * (h.abs() @ down.abs())
    # the bound of test_gpu_moe.py, whose 2^-13 stands for two chained sums of at most
    # 1024 terms, 2^-14 each; here the sums of a wave are longer, but what its matrix
    # instructions add is random in sign: n terms err by about sqrt(n) 2^-24 of their
    # root mean square, 2^-14 at n = 2^20
    assert bool(((Y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * mag).all())
