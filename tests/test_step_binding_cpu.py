"""The binding of the norm, the head's loss and the optimizer without a GPU:
tensors that only look like GPU tensors meet its checks, which all come before
any GPU call."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


class _Accepted(Exception):
    """Raised where a call, its arguments checked, asks for its workspace or for
    the library."""


@pytest.fixture
def q(monkeypatch):
    q = pytest.importorskip("bit_nf4_quantized_20_amd")

    def reached(*_):
        raise _Accepted
    monkeypatch.setattr(q, "_scratch", reached)
    monkeypatch.setattr(q, "_on", reached)
    return q


B16, F32, U8, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int64
T, H, V = 40, 192, 128


def _gpu(*shape, dtype=B16, dev="cuda:0"):
    return torch.empty(*shape, dtype=dtype, device=dev)


def _norm(q, **other):
    a = {"x": _gpu(T, H), "w": _gpu(H, dtype=F32), "res": _gpu(T, H), "h": _gpu(T, H), "y": _gpu(T, H), "rstd": _gpu(T, dtype=F32),
         "rows": q.FP8Rows(_gpu(T, 256, dtype=U8), _gpu(1, 256, 4, dtype=U8), T, H), "dy": _gpu(T, H), "dh": _gpu(T, H),
         "dw": _gpu(H, dtype=F32)}
    a.update(other)
    fwd = lambda: q.qlora_rmsnorm_fwd(a["x"], a["w"], residual=a["res"], h=a["h"], y=a["y"], rows=a["rows"], rstd=a["rstd"])
    bwd = lambda: q.qlora_rmsnorm_bwd(a["dy"], a["h"], a["w"], a["rstd"], dres=a["res"], dh=a["dh"], dweight=a["dw"])
    return fwd, bwd


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_norm(q):
    with FakeTensorMode():
        for call in _norm(q):
            with pytest.raises(_Accepted):
                call()
        for name, wrong, which in (
                ("x", _gpu(H, T), (0,)), ("x", _gpu(T, H, dtype=F32), (0,)), ("x", _gpu(T * H), (0,)), ("w", _gpu(H), (0, 1)),
                ("w", _gpu(H + 64, dtype=F32), (0, 1)), ("res", _gpu(T, H + 64), (0, 1)), ("h", _gpu(H, T), (0, 1)), ("y", _gpu(H, T), (0,)),
                ("rstd", _gpu(T + 1, dtype=F32), (0, 1)), ("dy", _gpu(T, H, dev="cuda:1"), (1,)), ("dh", _gpu(H, T), (1,)),
                ("dw", _gpu(H), (1,)), ("x", _gpu(H, T).t(), (0,)), ("x", torch.empty(T, H, dtype=B16, device="cpu"), (0,)),
                ("rows", q.FP8Rows(_gpu(T, 192, dtype=U8), _gpu(1, 256, 4, dtype=U8), T, H), (0,)),
                ("rows", q.FP8Rows(_gpu(T, 256, dtype=U8), _gpu(1, 40, 4, dtype=U8), T, H), (0,)),
                ("rows", q.FP8Rows(_gpu(T, 256, dtype=U8), _gpu(1, 256, 4, dtype=U8), T + 1, H), (0,)),
                ("rows", (1, 2), (0,)), ("x", None, (0,)), ("dy", None, (1,)), ("h", None, (1,))):
            calls = _norm(q, **{name: wrong})
            for c in which:
                with pytest.raises((TypeError, ValueError)):
                    calls[c]()
        x, w = _gpu(T, H), _gpu(H, dtype=F32)
        with pytest.raises(ValueError):  # no form of y
            q.qlora_rmsnorm_fwd(x, w, y16=False)
        with pytest.raises(ValueError):  # without a residual h is x
            q.qlora_rmsnorm_fwd(x, w, h=_gpu(T, H))
        with pytest.raises(_Accepted):
            q.qlora_rmsnorm_fwd(x, w, h=x)


def test_linear_from_rows(q):
    with FakeTensorMode():
        W = q.FP8Weight(_gpu(V, H, dtype=U8), _gpu(1, 2, dtype=U8), V, H)
        rows = lambda t=T, h=H: q.FP8Rows(_gpu(t, -(-h // 128) * 128, dtype=U8), _gpu(-(-h // 512), -(-t // 256) * 256, 4, dtype=U8), t, h)
        A, B = _gpu(8, H), _gpu(V, 8)
        for args in ((W, rows(), _gpu(T, H), A, B, 8, 16.0), (W, rows(), None, None, None, 0, 0.0)):
            with pytest.raises(_Accepted):
                q.qlora_fp8_linear_fwd_rows(*args)
        for args in ((W, rows(T + 1), _gpu(T, H), A, B, 8, 16.0), (W, rows(T, 256), None, None, None, 0, 0.0),
                     (W, rows(), _gpu(T, H + 64), A, B, 8, 16.0), (W, _gpu(T, H), None, None, None, 0, 0.0),
                     (W, rows(), _gpu(T, H), B, A, 8, 16.0)):
            with pytest.raises((TypeError, ValueError)):
                q.qlora_fp8_linear_fwd_rows(*args)


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_head(q):
    with FakeTensorMode():
        X, y, g = _gpu(T, H), _gpu(T, dtype=I64), _gpu(T, dtype=F32)
        n = V * H
        heads = {"bf16": _gpu(V, H), "fp8": q.FP8Weight(_gpu(V, H, dtype=U8), _gpu(1, 2, dtype=U8), V, H),
                 "nf4": q.NF4Weight(_gpu(n // 2, dtype=U8), _gpu(n // 64, dtype=U8), _gpu(-(-n // 16384), dtype=F32), V, H),
                 "nodq": q.NF4Weight(_gpu(n // 2, dtype=U8), None, _gpu(n // 64, dtype=F32), V, H, q.QLORA_NF4_ABSMAX_FP32)}
        for W in heads.values():
            for call in (lambda: q.qlora_head_loss(W, X, y), lambda: q.qlora_head_loss_grad(W, X, y, g)):
                with pytest.raises(_Accepted):
                    call()
        W = heads["bf16"]
        nf4 = lambda **k: q.NF4Weight(**{**heads["nf4"].__dict__, **k})
        for args in ((W, X, _gpu(T, dtype=torch.int32)), (W, X, _gpu(T + 1, dtype=I64)), (W, _gpu(T, H + 64), y), (W, X.float(), y),
                     (_gpu(V, H, dtype=F32), X, y), (_gpu(H, V).t(), X, y), (_gpu(V, H, dev="cuda:1"), X, y), (None, X, y), (W, None, y),
                     (nf4(codes=_gpu(n // 2 - 1, dtype=U8)), X, y), (nf4(absmax_q=None), X, y), (nf4(absmax_scale=_gpu(3, dtype=F32)), X, y),
                     (q.FP8Weight(_gpu(H, V, dtype=U8), _gpu(1, 2, dtype=U8), V, H), X, y),
                     (q.NF4Weight(heads["nodq"].codes, None, _gpu(n // 128, dtype=F32), V, H, q.QLORA_NF4_ABSMAX_FP32), X, y)):
            for call in (lambda: q.qlora_head_loss(*args), lambda: q.qlora_head_loss_grad(*args, g)):
                with pytest.raises((TypeError, ValueError)):
                    call()
        for kw in ({"loss": _gpu(T)}, {"lse": _gpu(T + 1, dtype=F32)}):
            with pytest.raises((TypeError, ValueError)):
                q.qlora_head_loss(W, X, y, **kw)


def test_adamw(q):
    with FakeTensorMode():
        p, f, g = _gpu(T, H), _gpu(T, H, dtype=F32), _gpu(T, H, dtype=F32)
        state = q.AdamWState(_gpu(T * H, dtype=F32), _gpu(T * H, dtype=F32))
        for bad in (([p], None, [g.double()], state), ([f], None, [g], state), (None, [p], [g], state), ([None], None, [g], state),
                    ([p, p], None, [g], state), ([p.t()], None, [g.t()], state), ([_gpu(H, T)], None, [g], state),
                    ([_gpu(T, H, dev="cuda:1")], None, [g], state), ([p], None, [torch.empty(T, H, device="cpu")], state),
                    ([p], None, [g], q.AdamWState(_gpu(T * H, dtype=F32), _gpu(T * H - 128, dtype=F32))),
                    ([p], None, [g], q.AdamWState(_gpu(T * H, dtype=U8), _gpu(T * H, dtype=U8), _gpu(60, dtype=U8), None)),
                    ([p], None, [g], (1, 2))):
            with pytest.raises((TypeError, ValueError)):
                q.qlora_adamw_plan(*bad)
        plan = q.AdamWPlan(state, 32, [0], [p, g], _gpu(256, dtype=U8), q._AdamWTableC())
        with pytest.raises((TypeError, ValueError)):
            q.qlora_adamw_step(plan, 1, lr=1e-3, grad_scale=_gpu(2, dtype=F32))
    assert q.qlora_adamw_state_len([1, 128, 129]) == 128 + 128 + 256
    with pytest.raises(q.QloraError):
        q.qlora_adamw_state_len([-1])
    s = q.qlora_adamw_state([5, 200], 8, "cpu")
    assert s.m.shape == s.v.shape == (384,) and s.m_scales.shape == (3,) and s.m.dtype == U8


def test_host_memory_is_refused(q):
    x, w, g = torch.zeros(4, 64, dtype=B16), torch.ones(64), torch.zeros(4, 64)
    for call in (lambda: q.qlora_rmsnorm_fwd(x, w), lambda: q.qlora_rmsnorm_bwd(x, x, w, torch.ones(4)),
                 lambda: q.qlora_head_loss(x, x, torch.zeros(4, dtype=I64)),
                 lambda: q.qlora_head_loss_grad(x, x, torch.zeros(4, dtype=I64), torch.ones(4)),
                 lambda: q.qlora_adamw_plan([x], None, [g], q.qlora_adamw_state([256], 32, "cpu")),
                 lambda: q.qlora_fp8_linear_fwd_rows(q.FP8Weight(torch.zeros(64, 64, dtype=U8), torch.zeros(1, 1, dtype=U8), 64, 64),
                                                     q.FP8Rows(torch.zeros(4, 128, dtype=U8), torch.zeros(1, 256, 4, dtype=U8), 4, 64),
                                                     x, None, None, 0, 0.0)):
        with pytest.raises(ValueError, match="a GPU is needed"):
            call()
