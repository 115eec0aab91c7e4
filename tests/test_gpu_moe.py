"""GPU parity of the mixture-of-experts operators against the fp64 oracle.

Ids are compared exactly.  Weights and logit gradients (fp32): every element
within 64 * 2^-24 of the magnitudes that enter it (an exponential is good to
2^-22, a sum of E <= 1024 terms takes at most 16 + 6 additions in a row, the
rest is a handful of products).  The expert layer: relative Frobenius <= 2e-3
(one rounding to bf16, 1.7e-3) and each element within 2^-8 of itself plus
2^-13 of the sum of its terms' magnitudes (two chained fp32 sums of at most
1024 terms, 2^-14 each at the very worst; the hidden values as hi + lo pairs,
2^-17, and the exponential, 2^-20, are below that)."""

import threading

import numpy as np
import pytest
import torch

import synth
from oracle import dense as odense
from oracle import moe as omoe
from oracle import native as onative
from oracle import nf4 as onf4

from gpu_util import TOL, banner, dev_bf16, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ router
def _route_case(q, l, k, renorm, dw):
    T, E = l.shape
    ids, w = q.qlora_moe_route(dev_f32(l), k, renormalize=renorm)
    rid, rw = omoe.route(l, k, renorm)
    assert ids.dtype == torch.int32 and np.array_equal(host(ids), rid)
    assert np.array_equal(np.isnan(host(w)), np.isnan(rw))
    ok = ~np.isnan(rw)
    assert (np.abs(host(w).astype(np.float64) - rw) <= 64 * 2.0 ** -24 * rw + 1e-37)[ok].all()
    dl = host(q.qlora_moe_route_bwd(dev_f32(l), ids, dev_f32(dw), renormalize=renorm)).astype(np.float64)
    fine = np.isfinite(rw).all(1)
    ref = omoe.route_bwd(l[fine], rid[fine], dw[fine], renorm)
    p = omoe.route_bwd(l[fine], rid[fine], np.zeros_like(dw[fine]), renorm)  # shapes only
    assert ref.shape == p.shape
    mag = 2.0 * np.abs(dw[fine]).max(axis=1, keepdims=True)
    share = np.zeros_like(ref)
    for i, row in enumerate(l[fine].astype(np.float64)):
        if not np.all(row == -np.inf):
            keep = np.isin(np.arange(E), rid[fine][i]) if renorm else np.ones(E, bool)
            x = np.where(keep, np.exp(row - row[keep].max()), 0)
            share[i] = x / x.sum()
    assert (np.abs(dl[fine] - ref) <= 64 * 2.0 ** -24 * mag * share + 1e-37).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 8, 8), (33, 16, 4), (5, 17, 16), (64, 60, 4),
                                   (301, 64, 6), (130, 128, 8), (9, 129, 3), (65, 256, 16), (3, 257, 1),
                                   (21, 1000, 16), (2, 1024, 8), (4099, 128, 8)])
def test_route_matches_oracle(T, E, k, renorm):
    q = require_gpu()
    banner(f"route T={T} E={E} k={k} renorm={renorm}")
    l = onf4.bf16_bits_to_f32(synth.bf16_bits(synth.normal_f32(T + E, (T, E), 1.5)))  # ties occur
    _route_case(q, l, k, renorm, synth.normal_f32(T + E + 1, (T, k), 1.0))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [6, 64, 200])
def test_route_special_rows(E, renorm):
    q = require_gpu()
    banner(f"route special rows E={E}")
    k = 4
    l = synth.normal_f32(3, (12, E), 1.0)
    low = np.finfo(np.float32).min
    l[0] = 0.0                                   # all equal
    l[1] = -np.inf                               # nothing may be chosen
    l[2, 1:] = -np.inf                           # one may
    l[3] = low                                   # all at the type's lowest value
    l[4, ::2] = low
    l[5, ::2], l[5, 1::2] = 0.0, -0.0            # the two zeros are equal
    l[6, 2] = np.nan
    l[7, 3] = np.inf
    l[8] = 1e38
    l[9] = np.linspace(-200, 200, E)             # exponentials that vanish
    l[10] = -1e38
    l[10, 5] = -9e37
    l[11, 0] = -np.inf
    _route_case(q, l.astype(np.float32), k, renorm, synth.normal_f32(4, (12, k), 1.0))


def test_route_bwd_takes_other_ids():
    # ids that are not the router's: outside [0, E) they are no choice
    q = require_gpu()
    banner("route bwd foreign ids")
    l = synth.normal_f32(5, (3, 20), 1.0)
    ids = np.array([[4, -1, 7], [19, 20, 0], [-5, 1000, -1]], dtype=np.int32)
    dw = synth.normal_f32(6, (3, 3), 1.0)
    for renorm in (True, False):
        got = host(q.qlora_moe_route_bwd(dev_f32(l), torch.from_numpy(ids).cuda(), dev_f32(dw), renormalize=renorm))
        for t in range(3):
            ok = (ids[t] >= 0) & (ids[t] < 20)
            if ok.any():
                ref = omoe.route_bwd(l[t:t + 1], ids[t:t + 1, ok], dw[t:t + 1, ok], renorm)
                assert np.abs(got[t] - ref).max() <= 1e-5
            else:
                assert not got[t].any()


# ------------------------------------------------------------------ experts
def _experts(q, seed, E, H, I):
    wg = synth.normal_f32(seed, (E * 2 * I, H), 1.0 / H ** 0.5)
    wd = synth.normal_f32(seed + 1, (E * H, I), 1.0 / I ** 0.5)
    gu, dn = q.nf4_quantize_weight(dev_f32(wg)), q.nf4_quantize_weight(dev_f32(wd))

    def values(w):
        return odense.widen(onf4.dequantize(*onf4.quantize(w.reshape(-1), nearest=onative.nearest_level)))
    return gu, dn, values(wg).reshape(E, 2, I, H), values(wd).reshape(E, H, I)


def _check(got_bits, ref, mag):
    got = onf4.bf16_bits_to_f32(got_bits).astype(np.float64)
    bad = np.abs(got - ref) > 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * mag
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])
    if ref.size >= 1024:
        assert odense.rel_frobenius(got, ref) <= TOL


@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 64, 64), (1, 8, 2, 128, 192), (1, 32, 8, 256, 128), (2, 8, 8, 64, 320), (3, 5, 2, 448, 64),
    (9, 8, 2, 512, 1024), (16, 16, 4, 1024, 256), (17, 2, 1, 192, 448), (33, 2, 2, 128, 128), (40, 60, 4, 320, 192),
    (64, 16, 8, 256, 320), (64, 3, 3, 128, 64), (32, 24, 16, 192, 128), (64, 1, 1, 128, 576),
])
def test_experts_match_oracle(T, E, k, H, I):
    q = require_gpu()
    banner(f"moe T={T} E={E} k={k} H={H} I={I}")
    gu, dn, vg, vd = _experts(q, 61, E, H, I)
    rng = np.random.Generator(np.random.PCG64(T + E))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.normal(0, 1, (T, k)).astype(np.float32)
    X = synth.bf16_bits(synth.normal_f32(62, (T, H), 1.0))
    big = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = q.qlora_moe_fwd(gu, dn, E, dev_bf16(X), torch.from_numpy(ids).cuda(), dev_f32(w), Y=big[:T])
    assert bool((big[T:] == 7.0).all())
    _check(host_bits(Y), *omoe.experts(vg, vd, odense.widen(X), ids, w))


@pytest.mark.parametrize("T,E,k,H,I", [
    (16, 64, 4, 1600, 512),   # tall row groups in both products
    (64, 16, 3, 2048, 1024),  # the same with two column tiles at a time
    (64, 2, 2, 256, 512),     # column tiles shared by several workgroups
    (4, 128, 8, 128, 1024),   # tall, then short; fewer pairs than experts
    (16, 32, 4, 256, 256), (16, 32, 4, 256, 320), (64, 8, 8, 512, 64), (61, 4, 4, 576, 256),
])
def test_experts_where_the_kernels_change(T, E, k, H, I):
    """Sizes that reach every kernel of the layer; the experts repeat five."""
    q = require_gpu()
    banner(f"moe borders T={T} E={E} k={k} H={H} I={I}")
    base = 5
    assert H * I % 16384 == 0  # an expert ends with a group of scales
    gu, dn, vg, vd = _experts(q, 65, base, H, I)
    which = torch.arange(E, device="cuda") % base

    def repeat(W):
        def pick(t):
            return t.view(base, -1)[which].reshape(-1).contiguous()
        return q.NF4Weight(pick(W.codes), pick(W.absmax_q), pick(W.absmax_scale), W.rows // base * E, W.cols)
    rng = np.random.Generator(np.random.PCG64(T * E + k))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[T // 2, 0] = -1
    w = rng.normal(0, 1, (T, k)).astype(np.float32)
    X = synth.bf16_bits(synth.normal_f32(66, (T, H), 1.0))
    Y = q.qlora_moe_fwd(repeat(gu), repeat(dn), E, dev_bf16(X), torch.from_numpy(ids).cuda(), dev_f32(w))
    _check(host_bits(Y), *omoe.experts(vg, vd, odense.widen(X), np.where(ids >= 0, ids % base, -1), w))


def test_experts_special_ids():
    q = require_gpu()
    banner("moe special ids")
    T, E, k, H, I = 40, 12, 4, 192, 256
    gu, dn, vg, vd = _experts(q, 71, E, H, I)
    rng = np.random.Generator(np.random.PCG64(9))
    ids = rng.integers(0, E, (T, k)).astype(np.int32)      # an expert may come twice in a row
    w = rng.normal(0, 1, (T, k)).astype(np.float32)
    ids[0] = -1                                            # no choice: 0
    ids[1] = [3, -1, E, 1 << 30]                           # one of four
    ids[2] = 5                                             # four times the same
    w[3] = 0.0
    ids[35:] = -1                                          # rows behind the last sequence
    X = synth.bf16_bits(synth.normal_f32(72, (T, H), 1.0))
    xd = dev_bf16(X)
    xd[35:] = float("nan")                                 # whose contents do not matter
    Y = host_bits(q.qlora_moe_fwd(gu, dn, E, xd, torch.from_numpy(ids).cuda(), dev_f32(w)))
    _check(Y, *omoe.experts(vg, vd, odense.widen(X), ids, w))
    assert not Y[0].any() and not Y[35:].any()
    # every pair at one expert: 160 columns
    ids[:] = 7
    Y = host_bits(q.qlora_moe_fwd(gu, dn, E, dev_bf16(X), torch.from_numpy(ids).cuda(), dev_f32(w)))
    _check(Y, *omoe.experts(vg, vd, odense.widen(X), ids, w))
    ids[:] = -1
    assert not host_bits(q.qlora_moe_fwd(gu, dn, E, dev_bf16(X), torch.from_numpy(ids).cuda(), dev_f32(w))).any()


def test_experts_rows_stay_their_own():
    q = require_gpu()
    banner("moe non-finite row")
    T, E, k, H, I = 20, 4, 2, 128, 128
    gu, dn, _, _ = _experts(q, 81, E, H, I)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    w = torch.rand(T, k, device="cuda")
    X = dev_bf16(synth.bf16_bits(synth.normal_f32(82, (T, H), 1.0)))
    clean = q.qlora_moe_fwd(gu, dn, E, X, ids, w)
    bad = X.clone()
    bad[4] = float("nan")
    Y = q.qlora_moe_fwd(gu, dn, E, bad, ids, w)
    keep = torch.arange(T, device="cuda") != 4
    assert torch.equal(Y[keep], clean[keep]) and bool(torch.isnan(Y[4]).all())


def test_binding_refuses_wrong_tensors():
    q = require_gpu()
    banner("moe binding refusals")
    T, E, k, H, I = 6, 4, 2, 128, 192
    gu, dn, _, _ = _experts(q, 83, E, H, I)
    X = dev_bf16(synth.bf16_bits(synth.normal_f32(84, (T, H), 1.0)))
    l = dev_f32(synth.normal_f32(85, (T, E), 1.0))
    ids, w = q.qlora_moe_route(l, k)
    ok = q.qlora_moe_fwd(gu, dn, E, X, ids, w)

    def refused(error, fn, *args, **kw):
        with pytest.raises(error):
            fn(*args, **kw)
    refused(q.QloraError, q.qlora_moe_route, l, 5)                                # k above the experts
    refused(q.QloraError, q.qlora_moe_route, l, 0)
    refused(ValueError, q.qlora_moe_route, dev_f32(synth.normal_f32(85, (E, T), 1.0)).t(), k)
    refused(TypeError, q.qlora_moe_route, l, k, ids=torch.empty(T, k, dtype=torch.int64, device="cuda"))
    refused(ValueError, q.qlora_moe_route_bwd, l, ids[:3], w)
    refused(TypeError, q.qlora_moe_route_bwd, l, ids.long(), w)
    refused(ValueError, q.qlora_moe_fwd, gu, dn, E, X[:, :64].contiguous(), ids, w)
    refused(ValueError, q.qlora_moe_fwd, gu, dn, E, X, ids[:3], w)
    refused(TypeError, q.qlora_moe_fwd, gu, dn, E, X, ids.long(), w)
    refused(q.QloraError, q.qlora_moe_fwd, gu, dn, E + 1, X, ids, w)              # not the weights' experts
    refused(ValueError, q.qlora_moe_fwd, dn, gu, E, X, ids, w)                    # the weights exchanged
    refused(ValueError, q.qlora_moe_fwd, gu, dn, E, X, ids, w, ws=torch.empty(1 << 20, dtype=torch.uint8))
    refused(q.QloraError, q.qlora_moe_fwd, gu, dn, E, X, ids, w, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    many = X.repeat(11, 1)
    refused(q.QloraError, q.qlora_moe_fwd, gu, dn, E, many, ids.repeat(11, 1), w.repeat(11, 1))  # 66 tokens
    assert torch.equal(q.qlora_moe_fwd(gu, dn, E, X, ids, w), ok)


def test_two_threads_on_one_stream():
    """Calls of two host threads whose launches interleave on the same stream."""
    q = require_gpu()
    banner("moe and fp8 from two threads")
    E, k, H, I, r, T = 8, 4, 256, 512, 16, 40
    gu, dn, _, _ = _experts(q, 86, E, H, I)
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(87, (H, H), 1.0 / H ** 0.5)))
    A = dev_bf16(synth.bf16_bits(synth.normal_f32(88, (r, H), 0.05)))
    B = dev_bf16(synth.bf16_bits(synth.normal_f32(89, (H, r), 0.05)))
    logits = dev_f32(synth.normal_f32(90, (T, E), 1.0))
    inputs = [dev_bf16(synth.bf16_bits(synth.normal_f32(91 + i, (T, H), 1.0))) for i in range(2)]

    def work(X):
        ids, w = q.qlora_moe_route(logits, k)
        return (*q.qlora_fp8_linear_bwd(W, X, X, A, B, r, 16.0), q.qlora_fp8_linear_fwd(W, X, A, B, r, 16.0),
                q.qlora_moe_fwd(gu, dn, E, X, ids, w))
    want = [work(X) for X in inputs]
    torch.cuda.synchronize()
    got = [[], []]

    def run(i):
        for _ in range(50):
            got[i].append(work(inputs[i]))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 50
        assert all(torch.equal(a, b) for out in got[i] for a, b in zip(out, want[i]))


def test_route_most_rows():
    """More rows than one launch takes (2^32 lanes)."""
    q = require_gpu()
    banner("route 2^29 rows")
    T = (1 << 29) + 7
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB of GPU memory")
    l = torch.zeros(T, 1, device="cuda")
    l[-1] = float("-inf")
    ids, w = q.qlora_moe_route(l, 1)
    assert not bool(ids.any()) and bool((w[:-1] == 1).all()) and w[-1].item() == 0
    l[-1] = 2.0
    w.fill_(3.0)
    assert not bool(q.qlora_moe_route_bwd(l, ids, w).any())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 6, 48])
def test_a_decode_block_eager_streams_and_graphs(T):
    """An 8-bit projection, the router and the experts as a decode step runs
    them, eager, on another stream, and captured twice and replayed between
    eager calls."""
    q = require_gpu()
    banner(f"moe block T={T}")
    E, k, H, I, r = 16, 4, 256, 192, 8
    gu, dn, vg, vd = _experts(q, 91, E, H, I)
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(93, (H, H), 1.0 / H ** 0.5)))
    A = dev_bf16(synth.bf16_bits(synth.normal_f32(94, (r, H), 0.05)))
    B = dev_bf16(synth.bf16_bits(synth.normal_f32(95, (H, r), 0.05)))
    gate = dev_f32(synth.normal_f32(96, (H, E), 0.1))
    X = dev_bf16(synth.bf16_bits(synth.normal_f32(97, (T, H), 1.0)))

    def block():
        h = q.qlora_fp8_linear_fwd(W, X, A, B, r, 16.0)
        logits = (h.float()[:, :, None] * gate[None]).sum(1)
        ids, w = q.qlora_moe_route(logits, k)
        return h, logits, ids, w, q.qlora_moe_fwd(gu, dn, E, h, ids, w)
    ref = [t.clone() for t in block()]
    rid, rw = omoe.route(host(ref[1]), k, True)
    assert np.array_equal(host(ref[2]), rid)
    _check(host_bits(ref[4]), *omoe.experts(vg, vd, odense.widen(host_bits(ref[0])), rid, rw))
    assert all(torch.equal(a, b) for a, b in zip(block(), ref))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = block()
        graphs.append((g, out))
    keep, other = X.clone(), dev_bf16(synth.bf16_bits(synth.normal_f32(98, (T, H), 1.0)))
    for turn in range(3):
        X.copy_(other if turn == 1 else keep)
        want = [t.clone() for t in block()]
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
