"""The norm on the GPU against oracle/norm.py in 64 bits, its 8-bit rows bit for
bit against oracle/fp8.py, and the 8-bit layer's forward from them.

u = 2^-24 is fp32's half step and 2^-8 bf16's, both relative to the value.  A sum of n
values of one sign is off by at most (its longest chain) u: a lane adds 8 C <= 32
squares, then at most 6 + 8 more additions, 46 u; the square root halves that, and
mean, sqrt, reciprocal add 4 u: rstd is within 2^-19."""

import numpy as np
import pytest
import torch

import synth
from oracle import fp8 as ofp8
from oracle import nf4 as onf4
from oracle import norm as onorm

from gpu_util import banner, dev_bf16, dev_f32, host, host_bits, require_gpu

pytestmark = pytest.mark.gpu

HALF16, RSTD, U = 2.0 ** -8, 2.0 ** -19, 2.0 ** -24
EPS = 1e-6
# each number of lanes a row and chunks a lane, next to its borders, rows that fill no workgroup
SIZES = [(1, 64), (5, 128), (37, 192), (33, 256), (18, 320), (17, 512), (9, 576), (5, 1024), (6, 1088), (7, 2048), (3, 2112),
         (4, 4096), (3, 4160), (2, 8192), (2, 8256), (2, 16384), (700, 64), (2100, 192), (600, 2048), (2300, 4160)]


def _wide(t):
    return onf4.bf16_bits_to_f32(host_bits(t)).astype(np.float64)


def _rows(seed, T, H):
    x = synth.normal_f32(seed, (T, H), 1.0) * np.exp(synth.normal_f32(seed + 1, (T, 1), 1.5))
    x[:, H // 3] *= 50
    return dev_bf16(synth.bf16_bits(x.astype(np.float32)))


def _weight(seed, H):
    return dev_f32(1 + 0.3 * synth.normal_f32(seed, (H,), 1.0))


def _check_rows8(y, rows, T, H):
    """Codes and scales of the 16-bit y, bit for bit; pads as documented."""
    yw = _wide(y)
    codes, scales = host(rows.codes), host(rows.scales)
    for c in range(0, H, 128):
        b = yw[:, c:c + 128]
        e = ofp8.scale_exponent(np.abs(b).max(axis=1))
        assert np.array_equal(scales[c // 512, :T, c // 128 % 4], (e + 127).astype(np.uint8)), c
        assert np.array_equal(codes[:, c:c + b.shape[1]], ofp8.encode(b / np.exp2(e.astype(np.float64))[:, None])), c
    assert not codes[:, H:].any()
    for b in range(-(-H // 128), 4 * -(-H // 512)):
        assert not scales[b // 4, :T, b % 4].any()


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("with_res", [True, False])
def test_forward(T, H, with_res):
    q = require_gpu()
    banner(f"norm forward {T}x{H} res={with_res}")
    x, w = _rows(100 + T + H, T, H), _weight(7 + H, H)
    res = _rows(300 + T + H, T, H) if with_res else None
    rows = q.FP8Rows(torch.full((T, -(-H // 128) * 128), 0x55, dtype=torch.uint8, device="cuda"),
                     torch.full((-(-H // 512), -(-T // 256) * 256, 4), 0x55, dtype=torch.uint8, device="cuda"), T, H)
    y, rows, h, rstd = q.qlora_rmsnorm_fwd(x, w, residual=res, eps=EPS, rows=rows)
    if with_res:
        exact = _wide(x) + _wide(res)
        assert (np.abs(_wide(h) - exact) <= HALF16 * (1 + 2.0 ** -14) * np.abs(exact)).all()
    else:
        assert h is x
    ry, rr = onorm.fwd(_wide(h), host(w).astype(np.float64), EPS)
    assert (np.abs(host(rstd) - rr) <= RSTD * rr).all()
    assert (np.abs(_wide(y) - ry) <= (HALF16 + 2 * RSTD) * np.abs(ry) + 1e-38).all()
    _check_rows8(y, rows, T, H)
    assert (host(rows.scales)[:, T:] == 0x55).all()  # behind the last row: as it was
    # the other forms of y are the same bits
    y2, none, _, _ = q.qlora_rmsnorm_fwd(x, w, residual=res, eps=EPS)
    assert none is None and torch.equal(y2, y)
    none, r8, _, _ = q.qlora_rmsnorm_fwd(x, w, residual=res, eps=EPS, y16=False, rows8=True)
    assert none is None and torch.equal(r8.codes, rows.codes) and torch.equal(r8.scales[:, :T], rows.scales[:, :T])


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("with_res,with_dw", [(True, True), (False, True), (True, False)])
def test_backward(T, H, with_res, with_dw):
    q = require_gpu()
    banner(f"norm backward {T}x{H} res={with_res} dw={with_dw}")
    h, w = _rows(500 + T + H, T, H), _weight(9 + H, H)
    _, _, _, rstd = q.qlora_rmsnorm_fwd(h, w, eps=EPS)
    dy = dev_bf16(synth.bf16_bits(synth.normal_f32(600 + T + H, (T, H), 1.0)))
    dres = dev_bf16(synth.bf16_bits(synth.normal_f32(700 + T + H, (T, H), 1.0))) if with_res else None
    need = q.qlora_rmsnorm_workspace_bytes(T, H)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    dh, dw = q.qlora_rmsnorm_bwd(dy, h, w, rstd, dres=dres, want_dweight=with_dw, ws=ws)
    rdh, rdw, mag, magw = onorm.bwd(_wide(dy), _wide(h), host(w).astype(np.float64), host(rstd).astype(np.float64),
                                    None if dres is None else _wide(dres))
    # the row's sum: a chain of at most 46 + 3 roundings of its magnitudes, six more behind it
    assert (np.abs(_wide(dh) - rdh) <= HALF16 * np.abs(rdh) + 64 * U * mag + 1e-38).all()
    if not with_dw:
        assert dw is None
        return
    # T terms of two roundings in some order: no chain is longer than T + 32
    assert (np.abs(host(dw) - rdw) <= (T + 34) * U * magw + 1e-38).all()
    again = q.qlora_rmsnorm_bwd(dy, h, w, rstd, dres=dres)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


def test_gradient_is_the_difference_of_the_forward():
    """dw against differences of sum(dy y): y is linear in w, so that only the
    roundings of y (2^-8 of each value, independent) and of dw count."""
    q = require_gpu()
    banner("norm differences")
    T, H = 40, 320
    h, w = _rows(801, T, H), _weight(802, H)
    dy = dev_bf16(synth.bf16_bits(synth.normal_f32(803, (T, H), 1.0)))
    y, _, _, rstd = q.qlora_rmsnorm_fwd(h, w, eps=EPS)
    dw = q.qlora_rmsnorm_bwd(dy, h, w, rstd)[1]
    for i in (0, 106, 319):
        up, dn = w.clone(), w.clone()
        up[i] += 0.5
        dn[i] -= 0.5
        f = [(q.qlora_rmsnorm_fwd(h, a, eps=EPS)[0][:, i].double() * dy[:, i].double()) for a in (up, dn)]
        bound = 5 * HALF16 * (f[0].norm() + f[1].norm()).item()
        assert abs((f[0].sum() - f[1].sum()).item() - dw[i].item()) <= bound


def test_outputs_over_inputs():
    """h may be x or the residual, dh may be dy or dres: the same bits."""
    q = require_gpu()
    banner("norm in place")
    for T, H in ((3, 192), (70, 2048), (5, 4160)):
        x, r, w, dy = _rows(1, T, H), _rows(2, T, H), _weight(3, H), _rows(4, T, H)
        y, _, h, rstd = q.qlora_rmsnorm_fwd(x, w, residual=r)
        for i in range(2):
            a, b = x.clone(), r.clone()
            y2, _, h2, _ = q.qlora_rmsnorm_fwd(a, w, residual=b, h=(a, b)[i])
            assert h2 is (a, b)[i] and torch.equal(h2, h) and torch.equal(y2, y)
        dh, dw = q.qlora_rmsnorm_bwd(dy, h, w, rstd, dres=r)
        for i in range(2):
            a, b = dy.clone(), r.clone()
            dh2, dw2 = q.qlora_rmsnorm_bwd(a, h, w, rstd, dres=b, dh=(a, b)[i])
            assert torch.equal(dh2, dh) and torch.equal(dw2, dw)


@pytest.mark.parametrize("H", [128, 576, 4160])
def test_rows_that_are_not_finite_stay_alone(H):
    q = require_gpu()
    banner(f"norm not finite H={H}")
    T = 9
    x, w, dy = _rows(11, T, H), _weight(12, H), _rows(13, T, H)
    y, rows, _, rstd = q.qlora_rmsnorm_fwd(x, w, rows8=True)
    dh, _ = q.qlora_rmsnorm_bwd(dy, x, w, rstd)
    bad = x.clone()
    bad[2, 5], bad[6, H - 1] = float("nan"), float("inf")
    yb, rb, _, sb = q.qlora_rmsnorm_fwd(bad, w, rows8=True)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[2] = keep[6] = False
    assert torch.equal(yb[keep], y[keep]) and torch.equal(rb.codes[keep], rows.codes[keep])
    assert torch.equal(rb.scales[:, :T][:, keep], rows.scales[:, :T][:, keep])
    assert bool(torch.isnan(yb[2]).all())
    # mean h^2 = inf, rstd = 0: 0 everywhere but at the infinity, whose product is NaN
    assert bool(torch.isnan(yb[6, H - 1])) and not bool(yb[6, :H - 1].any())
    dhb, dwb = q.qlora_rmsnorm_bwd(dy, bad, w, sb)
    assert torch.equal(dhb[keep], dh[keep]) and bool(torch.isnan(dhb[2]).all()) and bool(torch.isnan(dwb).any())
    # the layer behind it: a row of NaN, the others as ever
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(14, (192, H), 0.05)))
    xx, rr = torch.cat([bad, bad]), q.qlora_rmsnorm_fwd(torch.cat([bad, bad]), w, rows8=True)
    Y = q.qlora_fp8_linear_fwd_rows(W, rr[1], rr[0], None, None, 0, 0.0)
    assert bool(torch.isnan(Y[[2, 6, 11, 15]]).all()) and bool(torch.isfinite(Y[:T][keep]).all())
    # zero rows: rstd = 1 / sqrt(eps), y = 0; with eps = 0 0 times infinity
    zero = torch.zeros(2, H, dtype=torch.bfloat16, device="cuda")
    y0, r0, _, s0 = q.qlora_rmsnorm_fwd(zero, w, rows8=True, eps=EPS)
    assert not y0.any() and not r0.codes.any() and not r0.scales[:, :2].any() and np.allclose(host(s0), 1e3, rtol=1e-5)
    assert bool(torch.isnan(q.qlora_rmsnorm_fwd(zero, w, eps=0.0)[0]).all())


def test_more_rows_than_workgroups():
    """Rows behind the last workgroup's first are those of a call of their own."""
    q = require_gpu()
    T, H, n = 16500, 2112, 16300
    x, r, w = _rows(41, 200, H).repeat(83, 1)[:T].contiguous(), _rows(42, T, H), _weight(43, H)
    y, rows, h, rstd = q.qlora_rmsnorm_fwd(x, w, residual=r, rows8=True)
    z, tail, g, s = q.qlora_rmsnorm_fwd(x[n:], w, residual=r[n:], rows8=True)
    assert torch.equal(y[n:], z) and torch.equal(h[n:], g) and torch.equal(rstd[n:], s)
    assert torch.equal(rows.codes[n:], tail.codes) and torch.equal(rows.scales[:, n:T], tail.scales[:, :T - n])


def test_empty():
    q = require_gpu()
    banner("norm T=0")
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    w = _weight(1, 128)
    y, rows, h, rstd = q.qlora_rmsnorm_fwd(x, w, residual=x, rows8=True)
    assert y.shape == h.shape == (0, 128) and rstd.shape == (0,)
    dw = torch.full((128,), 3.0, device="cuda")
    dh, dw = q.qlora_rmsnorm_bwd(x, x, w, rstd, dweight=dw)
    assert not dw.any()


@pytest.mark.parametrize("T,H,n_out,r", [(1, 192, 128, 0), (16, 320, 192, 8), (17, 320, 192, 8), (40, 320, 192, 0), (64, 2048, 2112, 16),
                                         (300, 576, 192, 100), (300, 4160, 1088, 0), (3, 8256, 64, 4)])
def test_linear_from_rows(T, H, n_out, r):
    """The 8-bit layer on the norm's codes: the bits of the layer on its y."""
    q = require_gpu()
    banner(f"fp8 from rows T={T} {H}x{n_out} r={r}")
    W = q.qlora_fp8_quantize_weight(dev_f32(synth.normal_f32(21, (n_out, H), synth.W_STD)))
    A = dev_bf16(synth.bf16_bits(synth.normal_f32(22, (r, H), 0.05))) if r else None
    B = dev_bf16(synth.bf16_bits(synth.normal_f32(23, (n_out, r), 0.05))) if r else None
    y, rows, _, _ = q.qlora_rmsnorm_fwd(_rows(24, T, H), _weight(25, H), rows8=True)
    want = q.qlora_fp8_linear_fwd(W, y, A, B, r, 16.0)
    assert torch.equal(q.qlora_fp8_linear_fwd_rows(W, rows, y, A, B, r, 16.0), want)
    if r == 0 and (T > 16 or H > 8192):
        assert torch.equal(q.qlora_fp8_linear_fwd_rows(W, rows, None, None, None, 0, 0.0), want)
    elif r == 0:
        with pytest.raises(q.QloraError):
            q.qlora_fp8_linear_fwd_rows(W, rows, None, None, None, 0, 0.0)


def test_streams_graphs_and_other_shapes():
    q = require_gpu()
    banner("norm streams and graphs")
    T, H = 300, 576
    x, r, w, dy = _rows(31, T, H), _rows(32, T, H), _weight(33, H), _rows(34, T, H)

    def both():
        y, rows, h, rstd = q.qlora_rmsnorm_fwd(x, w, residual=r, rows8=True)
        dh, dw = q.qlora_rmsnorm_bwd(dy, h, w, rstd, dres=r)
        return y, rows.codes, rows.scales[:, :T], h, rstd, dh, dw
    ref = [t.clone() for t in both()]
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
    keep, other = x.clone(), _rows(35, T, H)
    for turn in range(3):
        x.copy_(other if turn == 1 else keep)
        want = [t.clone() for t in both()]
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
