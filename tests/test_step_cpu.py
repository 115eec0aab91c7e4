"""Norm, head loss and optimizer without a GPU: the oracle against autograd,
against differences and against its own definitions, and the library's refusals
(every check comes before any HIP call)."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import adamw as oadamw
from oracle import fp8 as ofp8
from oracle import head as ohead
from oracle import norm as onorm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.environ.get("QLORA_ABI_LIB") or os.path.join(ROOT, "bit_nf4_quantized_20_amd", "libqlora.so")
F = 0x10000  # 16-byte aligned address that is never dereferenced
ODD = 0x10008
NULL, SHAPE, ALIGN, WORKSPACE, VALUE = -1, -2, -3, -4, -7


# ------------------------------------------------------------------ oracle
def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _differences(f, x, grad, rng, h=1e-5, tol=1e-7, n=12):
    """Central differences at n places: error h^2 f''' / 6 and rounding 1e-16 f / h."""
    for _ in range(n):
        i = tuple(rng.integers(0, k) for k in x.shape)
        up, dn = x.copy(), x.copy()
        up[i] += h
        dn[i] -= h
        assert abs((f(up) - f(dn)) / (2 * h) - grad[i]) <= tol * (1 + abs(grad[i])), i


def test_norm_gradient_matches_differences_and_autograd():
    rng = _rng(1)
    h, w, G, R = rng.normal(0, 2, (5, 64)), rng.normal(1, .3, 64), rng.normal(0, 1, (5, 64)), rng.normal(0, 1, (5, 64))
    eps = 1e-3
    y, rstd = onorm.fwd(h, w, eps)
    dh, dw, _, _ = onorm.bwd(G, h, w, rstd, R)
    f = lambda h, w: float((G * onorm.fwd(h, w, eps)[0]).sum() + (R * h).sum())
    _differences(lambda a: f(a, w), h, dh, rng)
    _differences(lambda a: f(h, a), w, dw, rng)
    th, tw = torch.from_numpy(h).requires_grad_(True), torch.from_numpy(w).requires_grad_(True)
    ty = torch.nn.functional.rms_norm(th, (64,), tw, eps)
    assert np.allclose(ty.detach().numpy(), y, rtol=1e-12)
    ((ty * torch.from_numpy(G)).sum() + (th * torch.from_numpy(R)).sum()).backward()
    assert np.allclose(th.grad.numpy(), dh, rtol=1e-10) and np.allclose(tw.grad.numpy(), dw, rtol=1e-10)


def test_head_gradient_matches_differences_and_autograd():
    rng = _rng(2)
    X, W = rng.normal(0, 1, (6, 64)), rng.normal(0, .3, (37, 64))
    labels, g = np.array([3, 36, -100, 37, 0, 12]), rng.normal(0, 1, 6)
    X[5] = 40 * W[12]  # nearly sure
    loss, lse, dX, rest, mag = ohead.loss_grad(X, W, labels, g)
    assert not loss[2:4].any() and not dX[2:4].any() and 0 < rest[5] < 1e-6
    _differences(lambda a: float((g * ohead.loss_grad(a, W, labels)[0]).sum()), X, dX, rng, n=40)
    t = torch.from_numpy(X).requires_grad_(True)
    tl = torch.nn.functional.cross_entropy(t @ torch.from_numpy(W).t(), torch.from_numpy(np.where(labels == 37, -100, labels)),
                                           reduction="none", ignore_index=-100)
    assert np.allclose(tl.detach().numpy(), loss, rtol=1e-9, atol=1e-14)
    (tl * torch.from_numpy(g)).sum().backward()
    assert np.allclose(t.grad.numpy(), dX, rtol=1e-7, atol=1e-14)
    assert (np.abs(dX) <= mag * (1 + 1e-12)).all()


def test_adamw_matches_torch():
    rng = _rng(3)
    p0 = rng.normal(0, 1, 50)
    t = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    p, m, v = p0, np.zeros(50), np.zeros(50)
    for k in range(1, 6):
        g = rng.normal(0, 1, 50)
        t.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v = oadamw.step(p, g, m, v, k, 1e-2, 0.9, 0.99, 1e-8, 0.1)
        assert np.allclose(t.detach().numpy(), p, rtol=1e-12)


def test_rounding_with_noise_is_unbiased_and_keeps_codes():
    """Over all bytes of noise the mean of floor(y / d + (b + 1/2) / 256) is y / d up to
    1/512 (the grid of u); what is a code stays one."""
    rng = _rng(4)
    x = np.concatenate([rng.normal(0, 1, 100) * 10.0 ** rng.uniform(-5, 0, 100), [448.0], np.zeros(27)])
    y = oadamw.to8(x, np.full(128, 0.5), False)[2]
    d = oadamw.distance(y)
    mean = np.mean([np.abs(oadamw.to8(x, np.full(128, (b + .5) / 256), False)[0]) / d for b in range(256)], axis=0)
    assert (np.abs(mean - np.abs(y) / d) <= 1 / 512 + 1e-12).all()
    mags = ofp8.e4m3_values()[:127]
    x = np.concatenate([mags, [-448.0]])
    for u in (1 / 512, 511 / 512):
        val, sc, _, _ = oadamw.to8(x, np.full(128, u), False)
        assert np.array_equal(val, x) and sc[0] == 127
    # the rounded values are codes
    val = oadamw.to8(rng.normal(0, 1, 128), np.full(128, 0.9), False)[0]
    assert np.isin(np.abs(val), mags).all()
    # nothing that is not 0 becomes 0 where it must not
    small = np.zeros(128)
    small[0], small[1] = 1.0, 1e-12
    assert oadamw.to8(small, np.full(128, .1), True)[0][1] == 2.0 ** -9 and oadamw.to8(small, np.full(128, .1), False)[0][1] == 0


def test_noise_bytes_are_spread():
    um, ur = oadamw.noise(1 << 16, 7)
    for u in (um, ur):
        n = np.bincount((u * 256).astype(int), minlength=256)
        # 65536 draws over 256 bytes: mean 256, standard deviation 16
        assert n.min() > 256 - 6 * 16 and n.max() < 256 + 6 * 16
    assert abs(np.corrcoef(um, ur)[0, 1]) < 6 / 256 and abs(np.corrcoef(um[:-1], um[1:])[0, 1]) < 6 / 256
    other = oadamw.noise(1 << 16, 8)[0]
    assert abs(np.corrcoef(um, other)[0, 1]) < 6 / 256
    assert np.array_equal(oadamw.noise(64, 7, first=128)[0], um[128:192])


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.skip("libqlora.so not built")
    return ctypes.CDLL(LIB)


i64, p = ctypes.c_int64, ctypes.c_void_p
V = lambda a: None if a is None else p(a)


def _norm_fwd(lib, T=4, H=128, eps=1e-6, x=F, res=F, w=F, h=F, y=F, codes=F, scales=F, rstd=F):
    return lib.qlora_rmsnorm_fwd(V(x), V(res), V(w), i64(T), i64(H), ctypes.c_float(eps), V(h), V(y), V(codes), V(scales),
                                 V(rstd), None)


def test_norm_refusals(lib):
    assert [_norm_fwd(lib, **k) for k in ({"H": 0}, {"H": 96}, {"H": 16448}, {"T": -1}, {"T": 1 << 31}, {"H": -64})] == [SHAPE] * 6
    assert [_norm_fwd(lib, eps=e) for e in (-1e-9, float("nan"), float("inf"))] == [VALUE] * 3
    assert [_norm_fwd(lib, **{k: None}) for k in ("x", "w", "res", "h", "codes", "scales")] == [NULL] * 6
    assert _norm_fwd(lib, y=None, codes=None, scales=None) == NULL
    assert [_norm_fwd(lib, **{k: ODD}) for k in ("x", "res", "w", "h", "y", "codes", "scales")] == [ALIGN] * 7
    assert _norm_fwd(lib, rstd=F + 2) == ALIGN
    assert _norm_fwd(lib, T=0, x=None, w=None) == 0

    def bwd(T=4, H=128, dy=F, h=F, w=F, rstd=F, dres=F, dh=F, dw=F, ws=F, n=1 << 20):
        return lib.qlora_rmsnorm_bwd(V(dy), V(h), V(w), V(rstd), V(dres), i64(T), i64(H), V(dh), V(dw), V(ws),
                                     ctypes.c_size_t(n), None)
    assert [bwd(**k) for k in ({"H": 32}, {"T": -1}, {"H": 1 << 20})] == [SHAPE] * 3
    assert [bwd(**{k: None}) for k in ("dy", "h", "w", "rstd", "dh")] == [NULL] * 5
    assert [bwd(**{k: ODD}) for k in ("dy", "h", "w", "dres", "dh", "dw", "ws")] == [ALIGN] * 7
    assert bwd(rstd=F + 2) == ALIGN and bwd(rstd=F + 4, ws=None) == WORKSPACE
    lib.qlora_rmsnorm_workspace_bytes.restype = ctypes.c_size_t
    need = lib.qlora_rmsnorm_workspace_bytes(i64(4), i64(128))
    assert need >= 256 and bwd(n=need - 1) == WORKSPACE and bwd(ws=None) == WORKSPACE
    assert lib.qlora_rmsnorm_workspace_bytes(i64(4), i64(100)) == 0
    assert bwd(T=0, dw=None) == 0


def test_rows_refusals(lib):
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.qlora_fp8_rows_bytes(i64(3), i64(192), ctypes.byref(c), ctypes.byref(s)) == 0
    assert (c.value, s.value) == (3 * 256, 256 * 4)
    assert lib.qlora_fp8_rows_bytes(i64(257), i64(576), ctypes.byref(c), ctypes.byref(s)) == 0
    assert (c.value, s.value) == (257 * 640, 2 * 512 * 4)
    assert [lib.qlora_fp8_rows_bytes(i64(a), i64(b), None, None) for a, b in ((-1, 64), (1, 65), (1, -64), (1 << 31, 64))] == [SHAPE] * 4

    class W8(ctypes.Structure):
        _fields_ = [("codes", p), ("scales", p), ("rows", i64), ("cols", i64), ("flags", ctypes.c_uint32)]

    def fwd(T=40, codes=F, scales=F, X=F, A=F, B=F, r=8, n_in=192, n=1 << 30):
        w = W8(F, F, 128, n_in, 0)
        return lib.qlora_fp8_linear_fwd_rows(ctypes.byref(w), V(codes), V(scales), V(X), i64(T), V(A), V(B), i64(r),
                                             ctypes.c_float(16.0), V(F), V(F), ctypes.c_size_t(n), None)
    assert [fwd(**k) for k in ({"codes": None}, {"scales": None}, {"X": None}, {"A": None}, {"X": None, "r": 0, "T": 16})] == [NULL] * 5
    assert [fwd(**{k: ODD}) for k in ("codes", "scales", "X", "A", "B")] == [ALIGN] * 5
    # no X is needed: what is wrong next is the workspace
    assert fwd(X=None, r=0, n=16) == WORKSPACE and fwd(X=None, r=0, T=16, n_in=8256, n=16) == WORKSPACE
    assert fwd(T=0, codes=None, scales=None, X=None) == 0


class Nf4(ctypes.Structure):
    _fields_ = [("codes", p), ("q", p), ("scale", p), ("rows", i64), ("cols", i64), ("flags", ctypes.c_uint32)]


class Fp8(ctypes.Structure):
    _fields_ = [("codes", p), ("scales", p), ("rows", i64), ("cols", i64), ("flags", ctypes.c_uint32)]


class Head(ctypes.Structure):
    _fields_ = [("bf16", p), ("nf4", ctypes.POINTER(Nf4)), ("fp8", ctypes.POINTER(Fp8)), ("vocab", i64), ("hidden", i64)]


def test_head_refusals(lib):
    def call(head, T=4, X=F, labels=F, dloss=F, loss=F, lse=F, dX=F, ws=F, n=1 << 30, grad=True):
        args = [ctypes.byref(head) if head is not None else None, V(X), i64(T), V(labels)]
        if grad:
            return lib.qlora_head_loss_grad(*args, V(dloss), V(loss), V(lse), V(dX), V(ws), ctypes.c_size_t(n), None)
        return lib.qlora_head_loss(*args, V(loss), V(lse), V(ws), ctypes.c_size_t(n), None)

    def head(v=1000, h=128, **k):
        return Head(k.get("bf16", F), k.get("nf4"), k.get("fp8"), v, h)
    n4, f8 = Nf4(F, F, F, 640, 128, 0), Fp8(F, F, 640, 128, 0)
    ok4, ok8 = dict(bf16=None, nf4=ctypes.pointer(n4)), dict(bf16=None, fp8=ctypes.pointer(f8))
    for grad in (True, False):
        assert call(None, grad=grad) == NULL and call(head(bf16=None), grad=grad) == NULL
        assert call(head(640, nf4=ctypes.pointer(n4)), grad=grad) == VALUE
        assert [call(head(v, h), grad=grad) for v, h in ((0, 128), (-5, 128), ((1 << 24) + 1, 64), (10, 96), (10, 0), (10, 16448))] == [SHAPE] * 6
        assert [call(head(), T=t, grad=grad) for t in (-1, 1 << 31)] == [SHAPE] * 2
        assert [call(head(v, h, **k), grad=grad) for k in (ok4, ok8) for v, h in ((576, 128), (640, 192))] == [SHAPE] * 4
        assert [call(head(), grad=grad, **{k: None}) for k in ("X", "labels", "loss")] == [NULL] * 3
        assert [call(head(), grad=grad, **{k: ODD}) for k in ("X", "ws")] == [ALIGN] * 2
        assert [call(head(), grad=grad, **{k: F + 2}) for k in ("labels", "loss", "lse")] == [ALIGN] * 3
        assert call(head(), grad=grad, labels=F + 8, loss=F + 4, lse=F + 12, ws=None) == WORKSPACE
        assert call(head(bf16=ODD), grad=grad) == ALIGN
        assert call(head(), T=0, X=None, labels=None, grad=grad) == 0
        assert call(head(), ws=None, grad=grad) == WORKSPACE
        lib.qlora_head_workspace_bytes.restype = ctypes.c_size_t
        for k, v, expand in (({}, 1000, 0), (ok4, 640, 1), (ok8, 640, 1)):
            need = lib.qlora_head_workspace_bytes(i64(4), i64(v), i64(128), expand, int(grad))
            assert need > 256 and call(head(v, **k), n=need - 1, grad=grad) == WORKSPACE
    assert [call(head(), **{k: None}) for k in ("dloss", "dX")] == [NULL] * 2
    assert call(head(), dX=ODD) == ALIGN and call(head(), dloss=F + 2) == ALIGN
    bad = Nf4(F, F, F, 640, 128, 8)
    assert call(head(640, bf16=None, nf4=ctypes.pointer(bad))) == VALUE
    bad = Fp8(F, F, 640, 128, 1)
    assert call(head(640, bf16=None, fp8=ctypes.pointer(bad))) == VALUE
    assert lib.qlora_head_workspace_bytes(i64(4), i64(10), i64(96), 0, 0) == 0


def test_head_workspace_is_bounded(lib):
    """Rows go in rounds of at most 4096 and the vocabulary in pieces, so that the
    workspace does not grow with either."""
    lib.qlora_head_workspace_bytes.restype = ctypes.c_size_t
    w = lambda T, v, h, e, g: lib.qlora_head_workspace_bytes(i64(T), i64(v), i64(h), e, g)
    assert w(4096, 128000, 4096, 0, 1) < 512 << 20
    assert w(1 << 20, 1 << 24, 4096, 1, 1) < 1 << 30
    assert w(1 << 20, 128000, 4096, 0, 1) <= w(4096, 128000, 4096, 0, 1)
    assert w(4096, 1 << 24, 4096, 0, 0) <= 513 << 20
    # no rows: the smallest there is, no division by their number
    assert all(w(0, v, 64, e, g) >= 256 for v in (1, 1 << 24) for e in (0, 1) for g in (0, 1))


class Tensor(ctypes.Structure):
    _fields_ = [("param", p), ("master", p), ("grad", p), ("numel", i64)]


class Table(ctypes.Structure):
    _fields_ = [("table", p), ("chunks", i64), ("state_len", i64)]


class Rates(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [("step", i64), ("seed", ctypes.c_uint32)]


def test_adamw_refusals(lib):
    lib.qlora_adamw_state_len.restype = i64
    lib.qlora_adamw_table_bytes.restype = ctypes.c_size_t
    arr = lambda *n: (i64 * max(len(n), 1))(*n)
    assert lib.qlora_adamw_state_len(arr(1, 128, 129, 0), i64(4)) == 128 + 128 + 256
    assert lib.qlora_adamw_state_len(arr(), i64(0)) == 0
    assert [lib.qlora_adamw_state_len(arr(*n), i64(k)) for n, k in (((-1,), 1), (((1 << 32) + 1,), 1), ((1 << 32, 1), 2), ((1,), -1),
                                                                   ((1,), 65537))] == [-1] * 5
    assert lib.qlora_adamw_state_len(None, i64(1)) == -1
    assert lib.qlora_adamw_table_bytes(arr(-1), i64(1)) == 0 and lib.qlora_adamw_table_bytes(arr(2049), i64(1)) >= 256

    def plan(*ts, n=None, table=F, size=1 << 20, out=True):
        o = Table()
        a = (Tensor * max(len(ts), 1))(*ts)
        return lib.qlora_adamw_plan(a, i64(len(ts) if n is None else n), V(table), ctypes.c_size_t(size),
                                    ctypes.byref(o) if out else None, None)
    a = Tensor(0x100000, 0x200000, 0x300000, 1000)
    fine = lambda *ts: plan(*ts, size=16) == WORKSPACE  # all that comes before was accepted
    assert fine(a)
    assert [plan(a, n=k) for k in (-1, 65537)] == [SHAPE] * 2
    assert plan(a, table=None) == NULL and plan(a, out=False) == NULL and plan(a, table=ODD) == ALIGN
    assert plan(Tensor(None, None, F, 8)) == NULL and plan(Tensor(F, None, None, 8)) == NULL
    assert [plan(Tensor(ODD, None, F, 8)), plan(Tensor(None, ODD, F, 8)), plan(Tensor(F, None, ODD, 8))] == [ALIGN] * 3
    assert plan(Tensor(F, None, F + 4096, -1)) == SHAPE
    assert plan(Tensor(F, None, 0x300000, 5000), size=2 * 40) == WORKSPACE
    # the same memory twice: a parameter in two tensors, a master inside another, a gradient that is a parameter
    assert plan(a, a) == VALUE
    assert plan(a, Tensor(0x100000 + 1984, None, 0x400000, 8)) == VALUE
    assert fine(a, Tensor(0x100000 + 2000, None, 0x400000, 8))
    assert plan(a, Tensor(0x500000, 0x200000 + 3984, 0x400000, 8)) == VALUE
    assert plan(a, Tensor(0x500000, None, 0x200000 + 16, 8)) == VALUE
    assert plan(Tensor(F, F, 0x300000, 8)) == VALUE
    # one gradient for two tensors is read twice
    assert fine(a, Tensor(0x500000, None, 0x300000, 8))
    # nothing is asked of an empty tensor
    assert fine(Tensor(None, None, None, 0), a)

    def step(table=Table(F, 3, 6144), bits=8, m=F, v=F, ms=F, vs=F, gs=None, ok=True, **r):
        d = dict(lr=1e-3, beta1=.9, beta2=.999, eps=1e-8, weight_decay=0., step=1, seed=0)
        d.update(r)
        return lib.qlora_adamw_step(ctypes.byref(table) if table else None, bits, V(m), V(v), V(ms), V(vs), V(gs),
                                    ctypes.byref(Rates(**d)) if ok else None, None)
    nan, inf = float("nan"), float("inf")
    assert step(table=None) == NULL and step(ok=False) == NULL and step(table=Table(None, 3, 6144)) == NULL
    assert [step(bits=b) for b in (0, 4, 16, 64)] == [VALUE] * 4
    assert [step(**k) for k in ({"lr": nan}, {"lr": inf}, {"beta1": 1.}, {"beta1": -.1}, {"beta2": nan}, {"beta2": 1.}, {"eps": -1.},
                                {"eps": inf}, {"weight_decay": nan}, {"step": 0}, {"step": -3})] == [VALUE] * 11
    assert [step(**{k: None}) for k in ("m", "v", "ms", "vs")] == [NULL] * 4
    assert [step(**{k: ODD}) for k in ("m", "v", "ms", "vs")] == [ALIGN] * 4 and step(gs=F + 2) == ALIGN
    # states that share memory: 6144 elements and 48 scales each
    apart = dict(m=F, v=F + 6144, ms=F + 12288, vs=F + 12336)
    assert step(bits=32) == VALUE and step(bits=32, v=F + 6144) == VALUE
    assert [step(**{**apart, **k}) for k in ({"v": F + 6128}, {"m": F + 16}, {"ms": F + 12272}, {"vs": F + 12320}, {"vs": F + 12288})] == [VALUE] * 5
    assert step(table=Table(F, 3, -1)) == SHAPE
    assert step(table=Table(F, -1, 0)) == SHAPE and step(table=Table(F, 1 << 31, 0)) == SHAPE
    assert step(table=Table(F, 0, 0), m=None) == 0


def test_adamw_rates_that_fp32_does_not_hold(lib):
    def step(**r):
        d = dict(lr=1e-3, beta1=.9, beta2=.999, eps=1e-8, weight_decay=0., step=1, seed=0)
        d.update(r)
        t = Table(F, 0, 0)  # no tensors: what is accepted ends here
        return lib.qlora_adamw_step(ctypes.byref(t), 32, None, None, None, None, None, ctypes.byref(Rates(**d)), None)
    assert step() == 0 and step(eps=0.) == 0 and step(eps=1e-45) == 0 and step(lr=0., weight_decay=1e30) == 0
    assert step(eps=1e-46) == VALUE and step(eps=1e39) == VALUE
    assert step(lr=1e38) == VALUE and step(lr=1e38, beta1=0.) == 0 and step(lr=1e38, step=1000) == 0
    assert step(lr=1e20, weight_decay=-1e20) == VALUE and step(lr=-1e39, beta1=0.) == VALUE
