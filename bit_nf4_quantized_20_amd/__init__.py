"""Python binding of libqlora.so, the gfx950 NF4 / QLoRA-linear library.

Argument marshalling only: every step of the path runs in the library's HIP
kernels.  torch supplies device memory (``torch.empty``), raw pointers
(``data_ptr``) and the current stream; it computes nothing here.  If the
library has not been built, importing this package raises.

Names and semantics follow include/qlora.h:
    nf4_storage_bytes, nf4_quantize, nf4_dequantize, qlora_workspace_bytes,
    nf4_quantize_nodq, nf4_dequantize_nodq,
    qlora_linear_fwd, qlora_linear_bwd, qlora_workspace_bytes_multi, qlora_linear_fwd_multi,
    qlora_linear_bwd_multi, qlora_merge_workspace_bytes, qlora_merge,
    qlora_noalloc_scratch_bytes, qlora_linear_fwd_noalloc, qlora_workspace_bytes_flags,
    nf4_quantize_weight_nodq, nf4_code_buckets,
    qlora_fp8_storage_bytes, qlora_fp8_quantize, qlora_fp8_quantize_weight, qlora_fp8_dequantize,
    qlora_fp8_workspace_bytes, qlora_fp8_linear_fwd, qlora_fp8_linear_bwd, qlora_fp8_rows_bytes,
    qlora_fp8_linear_fwd_rows,
    qlora_moe_route, qlora_moe_route_bwd, qlora_moe_workspace_bytes, qlora_moe_fwd,
    qlora_rmsnorm_fwd, qlora_rmsnorm_workspace_bytes, qlora_rmsnorm_bwd,
    qlora_head_workspace_bytes, qlora_head_loss, qlora_head_loss_grad,
    qlora_adamw_state_len, qlora_adamw_state, qlora_adamw_plan, qlora_adamw_step,
    nf4_codebook, nf4_code_thresholds, qlora_status_string
"""

import ctypes
import functools
import os
import threading
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora.so")

QLORA_OK = 0
STATUS = {0: "OK", -1: "ERR_NULL", -2: "ERR_SHAPE", -3: "ERR_ALIGN", -4: "ERR_WORKSPACE",
          -5: "ERR_LAUNCH", -6: "ERR_DEVICE", -7: "ERR_VALUE"}


class QloraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_status_string(status)})")


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python bit_nf4_quantized_20_amd/build.py` "
                      "(hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)
_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t


class _NF4WeightC(ctypes.Structure):
    _fields_ = [("codes", _p), ("absmax_q", _p), ("absmax_scale", _p), ("rows", _i64),
                ("cols", _i64), ("flags", ctypes.c_uint32)]


QLORA_NF4_ABSMAX_FP32 = 0x1  # qlora_nf4_weight.flags: the 4.5-bit format (fp32 block absmax)


_lib.nf4_storage_bytes.argtypes = [_i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz), ctypes.POINTER(_sz)]
_lib.nf4_storage_bytes.restype = ctypes.c_int
_lib.nf4_quantize.argtypes = [_p, _i64, _p, _p, _p, _p]
_lib.nf4_quantize.restype = ctypes.c_int
_lib.nf4_dequantize.argtypes = [_p, _p, _p, _i64, _p, _p]
_lib.nf4_dequantize.restype = ctypes.c_int
_lib.qlora_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int]
_lib.qlora_workspace_bytes.restype = _sz
_lib.qlora_linear_fwd.argtypes = [ctypes.POINTER(_NF4WeightC), _p, _i64, _p, _p, _i64, ctypes.c_float,
                                  _p, _p, _sz, _p]
_lib.qlora_linear_fwd.restype = ctypes.c_int
_lib.qlora_linear_bwd.argtypes = [ctypes.POINTER(_NF4WeightC), _p, _p, _i64, _p, _p, _i64,
                                  ctypes.c_float, _p, _p, _p, _p, _sz, _p]
_lib.qlora_linear_bwd.restype = ctypes.c_int
_lib.qlora_workspace_bytes_multi.argtypes = [_i64, _i64, ctypes.POINTER(_i64), ctypes.c_int, _i64,
                                             ctypes.c_int]
_lib.qlora_workspace_bytes_multi.restype = _sz
_lib.qlora_linear_fwd_multi.argtypes = [ctypes.POINTER(_NF4WeightC), ctypes.c_int, _p, _i64,
                                        ctypes.POINTER(_p), ctypes.POINTER(_p), _i64, ctypes.c_float,
                                        _p, _p, _sz, _p]
_lib.qlora_linear_fwd_multi.restype = ctypes.c_int
_lib.qlora_linear_bwd_multi.argtypes = [ctypes.POINTER(_NF4WeightC), ctypes.c_int, _p, _p, _i64,
                                        ctypes.POINTER(_p), ctypes.POINTER(_p), _i64, ctypes.c_float,
                                        _p, ctypes.POINTER(_p), ctypes.POINTER(_p), _p, _sz, _p]
_lib.qlora_linear_bwd_multi.restype = ctypes.c_int
_lib.nf4_quantize_nodq.argtypes = [_p, _i64, _p, _p, _p]
_lib.nf4_quantize_nodq.restype = ctypes.c_int
_lib.nf4_dequantize_nodq.argtypes = [_p, _p, _i64, _p, _p]
_lib.nf4_dequantize_nodq.restype = ctypes.c_int
_lib.qlora_merge_workspace_bytes.argtypes = [_i64, _i64, _i64]
_lib.qlora_merge_workspace_bytes.restype = _sz
_lib.qlora_merge.argtypes = [ctypes.POINTER(_NF4WeightC), _p, _p, _i64, ctypes.c_float, _p, _p, _sz, _p]
_lib.qlora_merge.restype = ctypes.c_int
_lib.qlora_workspace_bytes_dropout.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int]
_lib.qlora_workspace_bytes_dropout.restype = _sz
_lib.qlora_linear_fwd_dropout.argtypes = [ctypes.POINTER(_NF4WeightC), _p, _i64, _p, ctypes.c_float, _p,
                                          _p, _i64, ctypes.c_float, _p, _p, _sz, _p]
_lib.qlora_linear_fwd_dropout.restype = ctypes.c_int
_lib.qlora_linear_bwd_dropout.argtypes = [ctypes.POINTER(_NF4WeightC), _p, _p, _i64, _p, ctypes.c_float,
                                          _p, _p, _i64, ctypes.c_float, _p, _p, _p, _p, _sz, _p]
_lib.qlora_linear_bwd_dropout.restype = ctypes.c_int
_lib.qlora_workspace_bytes_flags.argtypes = [_i64, _i64, ctypes.POINTER(_i64), ctypes.c_int, _i64, ctypes.c_int,
                                              ctypes.c_int, ctypes.c_uint32]
_lib.qlora_workspace_bytes_flags.restype = _sz
_lib.qlora_workspace_bytes_bwd_min.argtypes = [_i64, _i64, ctypes.POINTER(_i64), ctypes.c_int, _i64,
                                                ctypes.c_int, ctypes.c_uint32]
_lib.qlora_workspace_bytes_bwd_min.restype = _sz
_lib.qlora_workspace_bytes_fwd_min.argtypes = [_i64, _i64, ctypes.POINTER(_i64), ctypes.c_int, _i64,
                                                ctypes.c_int, ctypes.c_uint32]
_lib.qlora_workspace_bytes_fwd_min.restype = _sz
_lib.nf4_code_buckets.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_uint32)]
_lib.nf4_code_buckets.restype = None
_lib.qlora_noalloc_scratch_bytes.argtypes = []
_lib.qlora_noalloc_scratch_bytes.restype = _sz
_lib.qlora_linear_fwd_noalloc.argtypes = [ctypes.POINTER(_NF4WeightC), _p, _i64, _p, _p, _i64, ctypes.c_float,
                                          _p, _p]
_lib.qlora_linear_fwd_noalloc.restype = ctypes.c_int
_lib.nf4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
_lib.nf4_codebook.restype = None
_lib.nf4_code_thresholds.argtypes = [ctypes.POINTER(ctypes.c_float)]
_lib.nf4_code_thresholds.restype = None
_lib.qlora_status_string.argtypes = [ctypes.c_int]
_lib.qlora_status_string.restype = ctypes.c_char_p


class _FP8WeightC(ctypes.Structure):
    _fields_ = [("codes", _p), ("scales", _p), ("rows", _i64), ("cols", _i64), ("flags", ctypes.c_uint32)]


_lib.qlora_fp8_storage_bytes.argtypes = [_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]
_lib.qlora_fp8_storage_bytes.restype = ctypes.c_int
_lib.qlora_fp8_quantize.argtypes = [_p, _i64, _i64, _p, _p, _p]
_lib.qlora_fp8_quantize.restype = ctypes.c_int
_lib.qlora_fp8_dequantize.argtypes = [_p, _p, _i64, _i64, _p, _p]
_lib.qlora_fp8_dequantize.restype = ctypes.c_int
_lib.qlora_fp8_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int]
_lib.qlora_fp8_workspace_bytes.restype = _sz
_lib.qlora_fp8_linear_fwd.argtypes = [ctypes.POINTER(_FP8WeightC), _p, _i64, _p, _p, _i64, ctypes.c_float,
                                      _p, _p, _sz, _p]
_lib.qlora_fp8_linear_fwd.restype = ctypes.c_int
_lib.qlora_fp8_linear_bwd.argtypes = [ctypes.POINTER(_FP8WeightC), _p, _p, _i64, _p, _p, _i64, ctypes.c_float,
                                      _p, _p, _p, _p, _sz, _p]
_lib.qlora_fp8_linear_bwd.restype = ctypes.c_int
_lib.qlora_moe_route.argtypes = [_p, _i64, _i64, _i64, ctypes.c_int, _p, _p, _p]
_lib.qlora_moe_route.restype = ctypes.c_int
_lib.qlora_moe_route_bwd.argtypes = [_p, _p, _p, _i64, _i64, _i64, ctypes.c_int, _p, _p]
_lib.qlora_moe_route_bwd.restype = ctypes.c_int
_lib.qlora_moe_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64]
_lib.qlora_moe_workspace_bytes.restype = _sz
_lib.qlora_moe_fwd.argtypes = [ctypes.POINTER(_NF4WeightC), ctypes.POINTER(_NF4WeightC), _i64, _p, _i64, _p, _p,
                               _i64, _p, _p, _sz, _p]
_lib.qlora_moe_fwd.restype = ctypes.c_int
_lib.qlora_fp8_rows_bytes.argtypes = [_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]
_lib.qlora_fp8_rows_bytes.restype = ctypes.c_int
_lib.qlora_fp8_linear_fwd_rows.argtypes = [ctypes.POINTER(_FP8WeightC), _p, _p, _p, _i64, _p, _p, _i64, ctypes.c_float,
                                           _p, _p, _sz, _p]
_lib.qlora_fp8_linear_fwd_rows.restype = ctypes.c_int
_lib.qlora_rmsnorm_fwd.argtypes = [_p, _p, _p, _i64, _i64, ctypes.c_float, _p, _p, _p, _p, _p, _p]
_lib.qlora_rmsnorm_fwd.restype = ctypes.c_int
_lib.qlora_rmsnorm_workspace_bytes.argtypes = [_i64, _i64]
_lib.qlora_rmsnorm_workspace_bytes.restype = _sz
_lib.qlora_rmsnorm_bwd.argtypes = [_p, _p, _p, _p, _p, _i64, _i64, _p, _p, _p, _sz, _p]
_lib.qlora_rmsnorm_bwd.restype = ctypes.c_int


class _HeadC(ctypes.Structure):
    _fields_ = [("bf16", _p), ("nf4", ctypes.POINTER(_NF4WeightC)), ("fp8", ctypes.POINTER(_FP8WeightC)),
                ("vocab", _i64), ("hidden", _i64)]


_lib.qlora_head_workspace_bytes.argtypes = [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int]
_lib.qlora_head_workspace_bytes.restype = _sz
_lib.qlora_head_loss.argtypes = [ctypes.POINTER(_HeadC), _p, _i64, _p, _p, _p, _p, _sz, _p]
_lib.qlora_head_loss.restype = ctypes.c_int
_lib.qlora_head_loss_grad.argtypes = [ctypes.POINTER(_HeadC), _p, _i64, _p, _p, _p, _p, _p, _p, _sz, _p]
_lib.qlora_head_loss_grad.restype = ctypes.c_int


class _AdamWTensorC(ctypes.Structure):
    _fields_ = [("param", _p), ("master", _p), ("grad", _p), ("numel", _i64)]


class _AdamWTableC(ctypes.Structure):
    _fields_ = [("table", _p), ("chunks", _i64), ("state_len", _i64)]


class _AdamWRatesC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", _i64), ("seed", ctypes.c_uint32)]


_lib.qlora_adamw_state_len.argtypes = [ctypes.POINTER(_i64), _i64]
_lib.qlora_adamw_state_len.restype = _i64
_lib.qlora_adamw_table_bytes.argtypes = [ctypes.POINTER(_i64), _i64]
_lib.qlora_adamw_table_bytes.restype = _sz
_lib.qlora_adamw_plan.argtypes = [ctypes.POINTER(_AdamWTensorC), _i64, _p, _sz, ctypes.POINTER(_AdamWTableC), _p]
_lib.qlora_adamw_plan.restype = ctypes.c_int
_lib.qlora_adamw_step.argtypes = [ctypes.POINTER(_AdamWTableC), ctypes.c_int, _p, _p, _p, _p, _p,
                                  ctypes.POINTER(_AdamWRatesC), _p]
_lib.qlora_adamw_step.restype = ctypes.c_int


def _status_string(status: int) -> str:
    return _lib.qlora_status_string(int(status)).decode()


qlora_status_string = _status_string


def _check(status: int, where: str):
    if status != QLORA_OK:
        raise QloraError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: torch.Tensor, dtype, name: str, numel: int = None):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")


@dataclass
class NF4Weight:
    """Frozen NF4 weight [rows = out_features, cols = in_features].  flags 0:
    double-quantized (absmax_q uint8 per block, absmax_scale fp32 per 256
    blocks); QLORA_NF4_ABSMAX_FP32: the 4.5-bit format (absmax_q None,
    absmax_scale the fp32 absmax of each block)."""
    codes: torch.Tensor          # uint8 [rows*cols/2]
    absmax_q: torch.Tensor       # uint8 [rows*cols/64], or None (4.5-bit format)
    absmax_scale: torch.Tensor   # float32 [ceil(rows*cols/16384)], or [rows*cols/64]
    rows: int
    cols: int
    flags: int = 0

    def _c(self):
        q = None if self.absmax_q is None else self.absmax_q.data_ptr()
        return _NF4WeightC(self.codes.data_ptr(), q, self.absmax_scale.data_ptr(), self.rows, self.cols,
                           self.flags)


def nf4_storage_bytes(numel: int):
    c, q, s = _sz(), _sz(), _sz()
    _check(_lib.nf4_storage_bytes(numel, ctypes.byref(c), ctypes.byref(q), ctypes.byref(s)),
           "nf4_storage_bytes")
    return c.value, q.value, s.value


def nf4_quantize(w: torch.Tensor, codes=None, absmax_q=None, absmax_scale=None):
    """fp32 device tensor (any shape, numel % 64 == 0) -> (codes, absmax_q, absmax_scale)."""
    _need(w, torch.float32, "w")
    n = w.numel()
    cb, qb, sb = nf4_storage_bytes(n)
    dev = w.device
    if codes is None:
        codes = torch.empty(cb, dtype=torch.uint8, device=dev)
    if absmax_q is None:
        absmax_q = torch.empty(qb, dtype=torch.uint8, device=dev)
    if absmax_scale is None:
        absmax_scale = torch.empty(sb // 4, dtype=torch.float32, device=dev)
    _need(codes, torch.uint8, "codes", cb)
    _need(absmax_q, torch.uint8, "absmax_q", qb)
    _need(absmax_scale, torch.float32, "absmax_scale", sb // 4)
    _check(_lib.nf4_quantize(_ptr(w), n, _ptr(codes), _ptr(absmax_q), _ptr(absmax_scale),
                             _stream(dev)), "nf4_quantize")
    return codes, absmax_q, absmax_scale


def nf4_quantize_weight(w: torch.Tensor) -> NF4Weight:
    """Quantizes a [out, in] fp32 weight into an NF4Weight."""
    if w.dim() != 2:
        raise ValueError("weight must be 2-D [out, in]")
    c, q, s = nf4_quantize(w)
    return NF4Weight(c, q, s, w.shape[0], w.shape[1])


def nf4_quantize_weight_nodq(w: torch.Tensor) -> NF4Weight:
    """Quantizes a [out, in] fp32 weight into an NF4Weight of the 4.5-bit
    format (exact fp32 block absmax, no double quantization)."""
    if w.dim() != 2:
        raise ValueError("weight must be 2-D [out, in]")
    c, a = nf4_quantize_nodq(w)
    return NF4Weight(c, None, a, w.shape[0], w.shape[1], QLORA_NF4_ABSMAX_FP32)


def nf4_dequantize(codes, absmax_q, absmax_scale, numel: int, out=None):
    """-> bf16 device tensor [numel]."""
    if out is None:
        out = torch.empty(numel, dtype=torch.bfloat16, device=codes.device)
    _need(out, torch.bfloat16, "out", numel)
    _check(_lib.nf4_dequantize(_ptr(codes), _ptr(absmax_q), _ptr(absmax_scale), numel, _ptr(out),
                               _stream(codes.device)), "nf4_dequantize")
    return out


def nf4_quantize_nodq(w: torch.Tensor, codes=None, absmax=None):
    """fp32 device tensor (numel % 64 == 0) -> (codes uint8 [numel/2], absmax fp32 [numel/64]),
    no double quantization (4.5 bits per weight)."""
    _need(w, torch.float32, "w")
    n = w.numel()
    if codes is None:
        codes = torch.empty(n // 2, dtype=torch.uint8, device=w.device)
    if absmax is None:
        absmax = torch.empty(n // 64, dtype=torch.float32, device=w.device)
    _need(codes, torch.uint8, "codes", n // 2)
    _need(absmax, torch.float32, "absmax", n // 64)
    _check(_lib.nf4_quantize_nodq(_ptr(w), n, _ptr(codes), _ptr(absmax), _stream(w.device)),
           "nf4_quantize_nodq")
    return codes, absmax


def nf4_dequantize_nodq(codes, absmax, numel: int, out=None):
    """-> bf16 device tensor [numel] (fp32 block absmax, no double quantization)."""
    if out is None:
        out = torch.empty(numel, dtype=torch.bfloat16, device=codes.device)
    _need(out, torch.bfloat16, "out", numel)
    _check(_lib.nf4_dequantize_nodq(_ptr(codes), _ptr(absmax), numel, _ptr(out), _stream(codes.device)),
           "nf4_dequantize_nodq")
    return out


def qlora_workspace_bytes(T: int, in_features: int, out_features: int, r: int, backward: bool) -> int:
    return int(_lib.qlora_workspace_bytes(T, in_features, out_features, r, 1 if backward else 0))


_WS_CACHE = {}


def make_workspace(nbytes: int, device) -> torch.Tensor:
    """A workspace of at least nbytes (the library needs it uninitialised)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def qlora_workspace_bytes_flags(T: int, in_features: int, out_features, r: int, backward: bool,
                                dropout: bool = False, flags: int = 0) -> int:
    outs = (_i64 * len(out_features))(*[int(o) for o in out_features])
    return int(_lib.qlora_workspace_bytes_flags(T, in_features, outs, len(out_features), r,
                                                1 if backward else 0, 1 if dropout else 0, flags))


def qlora_workspace_bytes_fwd_min(T: int, in_features: int, out_features, r: int, dropout: bool = False,
                                  flags: int = 0) -> int:
    """The smallest forward workspace: no expanded W_hat (the GEMM then
    dequantizes the weight tiles while staging them)."""
    outs = (_i64 * len(out_features))(*[int(o) for o in out_features])
    return int(_lib.qlora_workspace_bytes_fwd_min(T, in_features, outs, len(out_features), r,
                                                  1 if dropout else 0, flags))


def qlora_workspace_bytes_bwd_min(T: int, in_features: int, out_features, r: int, dropout: bool = False,
                                  flags: int = 0) -> int:
    """The smallest backward workspace: no expanded W_hat^T (the dX GEMM then
    dequantizes the weight tiles while staging them)."""
    outs = (_i64 * len(out_features))(*[int(o) for o in out_features])
    return int(_lib.qlora_workspace_bytes_bwd_min(T, in_features, outs, len(out_features), r,
                                                  1 if dropout else 0, flags))


def _workspace(ws, T, n_in, n_out, r, backward, device, flags=0):
    """Caller's workspace, or a cached one per (device, stream) that grows as
    needed (concurrent streams get separate buffers)."""
    need = qlora_workspace_bytes_flags(T, n_in, [n_out], r, backward, False, flags)
    if ws is None:
        key = (torch.device(device).index, torch.cuda.current_stream(device).cuda_stream)
        ws = _WS_CACHE.get(key)
        if ws is None or ws.numel() < need:
            ws = make_workspace(need, device)
            _WS_CACHE[key] = ws
    return ws, ws.numel() * ws.element_size()


def qlora_linear_fwd(W: NF4Weight, X, A, B, r: int, alpha: float, Y=None, ws=None):
    """Y [T, out] bf16 = X W_hat^T + (alpha/r) (X A^T) B^T."""
    T = X.shape[0]
    _need(X, torch.bfloat16, "X", T * W.cols)
    _need(A, torch.bfloat16, "A", r * W.cols)
    _need(B, torch.bfloat16, "B", W.rows * r)
    if Y is None:
        Y = torch.empty(T, W.rows, dtype=torch.bfloat16, device=X.device)
    _need(Y, torch.bfloat16, "Y", T * W.rows)
    ws, ws_bytes = _workspace(ws, T, W.cols, W.rows, r, False, X.device, W.flags)
    wc = W._c()
    _check(_lib.qlora_linear_fwd(ctypes.byref(wc), _ptr(X), T, _ptr(A), _ptr(B), r, float(alpha),
                                 _ptr(Y), _ptr(ws), ws_bytes, _stream(X.device)), "qlora_linear_fwd")
    return Y


def qlora_noalloc_scratch_bytes() -> int:
    return int(_lib.qlora_noalloc_scratch_bytes())


def qlora_linear_fwd_noalloc(W: NF4Weight, X, A, B, r: int, alpha: float, Y):
    """qlora_linear_fwd on the library's static scratch: Y must be given (the
    call allocates nothing); calls that overlap on one GPU race."""
    T = X.shape[0]
    _need(X, torch.bfloat16, "X", T * W.cols)
    _need(A, torch.bfloat16, "A", r * W.cols)
    _need(B, torch.bfloat16, "B", W.rows * r)
    _need(Y, torch.bfloat16, "Y", T * W.rows)
    wc = W._c()
    _check(_lib.qlora_linear_fwd_noalloc(ctypes.byref(wc), _ptr(X), T, _ptr(A), _ptr(B), r, float(alpha),
                                         _ptr(Y), _stream(X.device)), "qlora_linear_fwd_noalloc")
    return Y


def qlora_linear_bwd(W: NF4Weight, X, dY, A, B, r: int, alpha: float, dX=None, dA=None, dB=None,
                     ws=None):
    """-> (dX [T, in] bf16, dA [r, in] fp32, dB [out, r] fp32)."""
    T = X.shape[0]
    _need(X, torch.bfloat16, "X", T * W.cols)
    _need(dY, torch.bfloat16, "dY", T * W.rows)
    _need(A, torch.bfloat16, "A", r * W.cols)
    _need(B, torch.bfloat16, "B", W.rows * r)
    dev = X.device
    if dX is None:
        dX = torch.empty(T, W.cols, dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty(r, W.cols, dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty(W.rows, r, dtype=torch.float32, device=dev)
    _need(dX, torch.bfloat16, "dX", T * W.cols)
    _need(dA, torch.float32, "dA", r * W.cols)
    _need(dB, torch.float32, "dB", W.rows * r)
    ws, ws_bytes = _workspace(ws, T, W.cols, W.rows, r, True, dev, W.flags)
    wc = W._c()
    _check(_lib.qlora_linear_bwd(ctypes.byref(wc), _ptr(X), _ptr(dY), T, _ptr(A), _ptr(B), r,
                                 float(alpha), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws_bytes,
                                 _stream(dev)), "qlora_linear_bwd")
    return dX, dA, dB


def qlora_workspace_bytes_dropout(T: int, in_features: int, out_features: int, r: int,
                                  backward: bool) -> int:
    return int(_lib.qlora_workspace_bytes_dropout(T, in_features, out_features, r, 1 if backward else 0))


def _dropout_ws(ws, T, n_in, n_out, r, backward, device, flags=0):
    need = qlora_workspace_bytes_flags(T, n_in, [n_out], r, backward, True, flags)
    if ws is None:
        key = (torch.device(device).index, torch.cuda.current_stream(device).cuda_stream)
        ws = _WS_CACHE.get(key)
        if ws is None or ws.numel() < need:
            ws = make_workspace(need, device)
            _WS_CACHE[key] = ws
    return ws, ws.numel() * ws.element_size()


def qlora_linear_fwd_dropout(W: NF4Weight, X, keep, p: float, A, B, r: int, alpha: float, Y=None,
                             ws=None):
    """Y = X W_hat^T + (alpha/r) ((keep o X / (1 - p)) A^T) B^T; keep is the
    packed mask [T, in/8] uint8 (bit k % 8 of byte k / 8 = element k kept)."""
    T = X.shape[0]
    _need(X, torch.bfloat16, "X", T * W.cols)
    _need(keep, torch.uint8, "keep", T * (W.cols // 8))
    _need(A, torch.bfloat16, "A", r * W.cols)
    _need(B, torch.bfloat16, "B", W.rows * r)
    if Y is None:
        Y = torch.empty(T, W.rows, dtype=torch.bfloat16, device=X.device)
    _need(Y, torch.bfloat16, "Y", T * W.rows)
    ws, ws_bytes = _dropout_ws(ws, T, W.cols, W.rows, r, False, X.device, W.flags)
    wc = W._c()
    _check(_lib.qlora_linear_fwd_dropout(ctypes.byref(wc), _ptr(X), T, _ptr(keep), float(p), _ptr(A),
                                         _ptr(B), r, float(alpha), _ptr(Y), _ptr(ws), ws_bytes,
                                         _stream(X.device)), "qlora_linear_fwd_dropout")
    return Y


def qlora_linear_bwd_dropout(W: NF4Weight, X, dY, keep, p: float, A, B, r: int, alpha: float, dX=None,
                             dA=None, dB=None, ws=None):
    """Backward of qlora_linear_fwd_dropout with the same mask ->
    (dX [T, in] bf16, dA [r, in] fp32, dB [out, r] fp32)."""
    T = X.shape[0]
    _need(X, torch.bfloat16, "X", T * W.cols)
    _need(dY, torch.bfloat16, "dY", T * W.rows)
    _need(keep, torch.uint8, "keep", T * (W.cols // 8))
    _need(A, torch.bfloat16, "A", r * W.cols)
    _need(B, torch.bfloat16, "B", W.rows * r)
    dev = X.device
    if dX is None:
        dX = torch.empty(T, W.cols, dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty(r, W.cols, dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty(W.rows, r, dtype=torch.float32, device=dev)
    _need(dX, torch.bfloat16, "dX", T * W.cols)
    _need(dA, torch.float32, "dA", r * W.cols)
    _need(dB, torch.float32, "dB", W.rows * r)
    ws, ws_bytes = _dropout_ws(ws, T, W.cols, W.rows, r, True, dev, W.flags)
    wc = W._c()
    _check(_lib.qlora_linear_bwd_dropout(ctypes.byref(wc), _ptr(X), _ptr(dY), T, _ptr(keep), float(p),
                                         _ptr(A), _ptr(B), r, float(alpha), _ptr(dX), _ptr(dA), _ptr(dB),
                                         _ptr(ws), ws_bytes, _stream(dev)), "qlora_linear_bwd_dropout")
    return dX, dA, dB


def qlora_merge_workspace_bytes(in_features: int, out_features: int, r: int) -> int:
    return int(_lib.qlora_merge_workspace_bytes(in_features, out_features, r))


def qlora_merge(W: NF4Weight, A, B, r: int, alpha: float, out=None, ws=None):
    """W_merged [out, in] bf16 = bf16(W_hat + (alpha/r) B A)."""
    _need(A, torch.bfloat16, "A", r * W.cols)
    _need(B, torch.bfloat16, "B", W.rows * r)
    dev = A.device
    if out is None:
        out = torch.empty(W.rows, W.cols, dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", W.rows * W.cols)
    need = qlora_merge_workspace_bytes(W.cols, W.rows, r)
    if ws is None:
        ws = make_workspace(need, dev)
    wc = W._c()
    _check(_lib.qlora_merge(ctypes.byref(wc), _ptr(A), _ptr(B), r, float(alpha), _ptr(out), _ptr(ws),
                            ws.numel() * ws.element_size(), _stream(dev)), "qlora_merge")
    return out


def qlora_workspace_bytes_multi(T: int, in_features: int, out_features, r: int, backward: bool) -> int:
    outs = (_i64 * len(out_features))(*[int(o) for o in out_features])
    return int(_lib.qlora_workspace_bytes_multi(T, in_features, outs, len(out_features), r,
                                                1 if backward else 0))


def _multi_ws(ws, T, n_in, outs, r, backward, device, flags=0):
    need = qlora_workspace_bytes_flags(T, n_in, outs, r, backward, False, flags)
    if ws is None:
        ws = make_workspace(need, device)
    return ws, ws.numel() * ws.element_size()


def _ptr_array(ts):
    return (_p * len(ts))(*[t.data_ptr() for t in ts])


def qlora_linear_fwd_multi(Ws, X, As, Bs, r: int, alpha: float, Y=None, ws=None):
    """Projections sharing X (e.g. q|k|v, gate|up): Y [T, sum out_i] bf16 with
    projection i's columns side by side."""
    n = len(Ws)
    T = X.shape[0]
    n_in = Ws[0].cols
    outs = [W.rows for W in Ws]
    _need(X, torch.bfloat16, "X", T * n_in)
    for W, A, B in zip(Ws, As, Bs):
        _need(A, torch.bfloat16, "A", r * W.cols)
        _need(B, torch.bfloat16, "B", W.rows * r)
    if Y is None:
        Y = torch.empty(T, sum(outs), dtype=torch.bfloat16, device=X.device)
    _need(Y, torch.bfloat16, "Y", T * sum(outs))
    ws, ws_bytes = _multi_ws(ws, T, n_in, outs, r, False, X.device, Ws[0].flags)
    wc = (_NF4WeightC * n)(*[W._c() for W in Ws])
    _check(_lib.qlora_linear_fwd_multi(wc, n, _ptr(X), T, _ptr_array(As), _ptr_array(Bs), r,
                                       float(alpha), _ptr(Y), _ptr(ws), ws_bytes, _stream(X.device)),
           "qlora_linear_fwd_multi")
    return Y


def qlora_linear_bwd_multi(Ws, X, dY, As, Bs, r: int, alpha: float, dX=None, dAs=None, dBs=None,
                           ws=None):
    """-> (dX [T, in] bf16 summed over the projections, [dA_i fp32], [dB_i fp32])."""
    n = len(Ws)
    T = X.shape[0]
    n_in = Ws[0].cols
    outs = [W.rows for W in Ws]
    dev = X.device
    _need(X, torch.bfloat16, "X", T * n_in)
    _need(dY, torch.bfloat16, "dY", T * sum(outs))
    if dX is None:
        dX = torch.empty(T, n_in, dtype=torch.bfloat16, device=dev)
    if dAs is None:
        dAs = [torch.empty(r, n_in, dtype=torch.float32, device=dev) for _ in range(n)]
    if dBs is None:
        dBs = [torch.empty(o, r, dtype=torch.float32, device=dev) for o in outs]
    ws, ws_bytes = _multi_ws(ws, T, n_in, outs, r, True, dev, Ws[0].flags)
    wc = (_NF4WeightC * n)(*[W._c() for W in Ws])
    _check(_lib.qlora_linear_bwd_multi(wc, n, _ptr(X), _ptr(dY), T, _ptr_array(As), _ptr_array(Bs),
                                       r, float(alpha), _ptr(dX), _ptr_array(dAs), _ptr_array(dBs),
                                       _ptr(ws), ws_bytes, _stream(dev)), "qlora_linear_bwd_multi")
    return dX, dAs, dBs


def nf4_codebook():
    out = (ctypes.c_float * 16)()
    _lib.nf4_codebook(out)
    return [float(v) for v in out]


def nf4_code_buckets():
    """-> (thr [33], base [33]): the quantize kernel's code lookup on X = 16 x."""
    thr, base = (ctypes.c_float * 33)(), (ctypes.c_uint32 * 33)()
    _lib.nf4_code_buckets(thr, base)
    return [float(v) for v in thr], [int(v) for v in base]


def nf4_code_thresholds():
    out = (ctypes.c_float * 15)()
    _lib.nf4_code_thresholds(out)
    return [float(v) for v in out]


# ---------------------------------------------------------------------------
# The 8-bit linear layer and the mixture-of-experts operators.  Every tensor of
# a call lies on one GPU, which becomes the current one for the call; the work
# goes to that GPU's current stream.
# ---------------------------------------------------------------------------
@dataclass
class FP8Weight:
    """Frozen 8-bit weight [rows = out_features, cols = in_features]: e4m3
    codes, one power-of-two scale byte per 128 x 128 block."""
    codes: torch.Tensor   # uint8 [rows, cols]
    scales: torch.Tensor  # uint8 [ceil(rows/128), ceil(cols/128)]
    rows: int
    cols: int

    def _c(self):
        return _FP8WeightC(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols, 0)


def _arg(t, dtype, shape, name: str, dev, index: int = None):
    """A contiguous tensor of this type, device and size (shape: its sizes, or
    its element count); index: its place in a list.  One chain of tests for the call that is right; what
    is wrong is found out afterwards."""
    if (t is not None and t.dtype is dtype and t.device == dev and t.is_contiguous() and dev.type == "cuda"
            and (t.numel() == shape if type(shape) is int else t.shape == shape)):
        return
    if index is not None:
        name = f"{name}[{index}]"
    _arg_rest(t, dtype, name, dev)
    raise ValueError(f"{name}: expected {tuple(shape) if type(shape) is torch.Size else shape} elements, got {tuple(t.shape)}")


def _rows_arg(t, dtype, rows: int, cols: int, name: str, dev):
    """As _arg, once the call's first tensor has shown that dev is a GPU, for a
    row-major matrix: [rows, cols], the same rows under more axes, or flat.  A
    transposed one has the right number of elements and would be read or
    written in the wrong order."""
    if (t is not None and t.dtype is dtype and t.device == dev and t.is_contiguous()
            and (t.shape == (rows, cols)
                 or t.numel() == rows * cols and t.dim() > 0 and (t.dim() == 1 or t.shape[-1] == cols))):
        return
    _arg_rest(t, dtype, name, dev)
    raise ValueError(f"{name}: expected ({rows}, {cols}), got {tuple(t.shape)}")


def _arg_rest(t, dtype, name: str, dev):
    """Raises for what is wrong besides the size."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != dev or dev.type != "cuda":
        raise ValueError(f"{name}: on {t.device}, the call runs on {dev} (a GPU is needed)")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _matrix(t, name: str):
    """(rows, cols) of a 2-D tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dim() != 2:
        raise ValueError(f"{name}: must be 2-D, got {t.dim()}-D")
    return t.shape


# the current stream's handle by device index (the public query builds a
# Stream object, 1.9 us against 0.1 of a call's 8); the current GPU and whether its
# current stream is being captured (0.2 and 0.3 us against 0.1 and 0.2)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_captures = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _on(dev, fn, where: str, *args):
    """Calls fn(*args, stream) with dev current, on dev's current stream."""
    index = dev.index
    if _current_gpu() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(index))
    if st != QLORA_OK:
        raise QloraError(st, where)


_SCRATCH = threading.local()


def _capturing(dev) -> bool:
    """Whether dev's current stream is being captured (torch asks about the
    current GPU's)."""
    if _current_gpu() == dev.index:
        return _captures()
    with torch.cuda.device(dev):
        return _captures()


# the most bytes of a workspace that is kept: a larger one comes from torch's
# allocator and goes back to it (1.3 us, where such a call's kernels take 20 and
# more)
_KEEP_MOST = 32 << 20


def _scratch(ws, need: int, dev):
    """The caller's workspace, or one kept per host thread, device and stream
    (the launches of two threads' calls may interleave on one stream).  Under
    graph capture it is a new allocation of the graph's own pool: a replay then
    shares no scratch with eager calls or with other graphs."""
    if ws is None:
        if need > _KEEP_MOST or _capturing(dev):
            ws = make_workspace(need, dev)
        else:
            kept = _SCRATCH.__dict__
            key = (dev.index, _raw_stream(dev.index))
            ws = kept.get(key)
            if ws is None or ws.numel() < need:
                kept[key] = ws = make_workspace(need, dev)
    elif ws.device != dev:
        raise ValueError(f"ws: on {ws.device}, the call runs on {dev}")
    elif not ws.is_contiguous():
        raise ValueError("ws: must be contiguous")
    return ws


@functools.lru_cache(maxsize=4096)
def qlora_fp8_storage_bytes(rows: int, cols: int):
    c, s = _sz(), _sz()
    _check(_lib.qlora_fp8_storage_bytes(rows, cols, ctypes.byref(c), ctypes.byref(s)), "qlora_fp8_storage_bytes")
    return c.value, s.value


def qlora_fp8_quantize(w: torch.Tensor, codes=None, scales=None):
    """fp32 device tensor [rows, cols] (multiples of 64) -> (codes uint8 [rows,
    cols], scales uint8 [ceil(rows/128), ceil(cols/128)])."""
    rows, cols = _matrix(w, "w")
    dev = w.device
    _arg(w, torch.float32, rows * cols, "w", dev)
    qlora_fp8_storage_bytes(rows, cols)  # refuses other sizes
    grid = (-(-rows // 128), -(-cols // 128))
    if codes is None:
        codes = torch.empty(rows, cols, dtype=torch.uint8, device=dev)
    else:
        _rows_arg(codes, torch.uint8, rows, cols, "codes", dev)
    if scales is None:
        scales = torch.empty(grid, dtype=torch.uint8, device=dev)
    else:
        _rows_arg(scales, torch.uint8, *grid, "scales", dev)
    _on(dev, _lib.qlora_fp8_quantize, "qlora_fp8_quantize", w.data_ptr(), rows, cols, codes.data_ptr(),
        scales.data_ptr())
    return codes, scales


def qlora_fp8_quantize_weight(w: torch.Tensor) -> FP8Weight:
    """Quantizes a [out, in] fp32 weight into an FP8Weight."""
    codes, scales = qlora_fp8_quantize(w)
    return FP8Weight(codes, scales, w.shape[0], w.shape[1])


def qlora_fp8_dequantize(codes, scales, rows: int, cols: int, out=None):
    """-> bf16 device tensor [rows, cols]."""
    dev = codes.device
    qlora_fp8_storage_bytes(rows, cols)  # refuses other sizes
    if dev.type != "cuda":
        _arg_rest(codes, torch.uint8, "codes", dev)
    _rows_arg(codes, torch.uint8, rows, cols, "codes", dev)
    _rows_arg(scales, torch.uint8, -(-rows // 128), -(-cols // 128), "scales", dev)
    if out is None:
        out = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    else:
        _rows_arg(out, torch.bfloat16, rows, cols, "out", dev)
    _on(dev, _lib.qlora_fp8_dequantize, "qlora_fp8_dequantize", codes.data_ptr(), scales.data_ptr(), rows, cols,
        out.data_ptr())
    return out


@functools.lru_cache(maxsize=4096)
def qlora_fp8_workspace_bytes(T: int, in_features: int, out_features: int, r: int, backward: bool) -> int:
    return int(_lib.qlora_fp8_workspace_bytes(T, in_features, out_features, r, 1 if backward else 0))


def _fp8_args(W, A, B, r, dev):
    _rows_arg(W.codes, torch.uint8, W.rows, W.cols, "W.codes", dev)
    _rows_arg(W.scales, torch.uint8, -(-W.rows // 128), -(-W.cols // 128), "W.scales", dev)
    if r > 0:
        _rows_arg(A, torch.bfloat16, r, W.cols, "A", dev)
        _rows_arg(B, torch.bfloat16, W.rows, r, "B", dev)


def qlora_fp8_linear_fwd(W: FP8Weight, X, A, B, r: int, alpha: float, Y=None, ws=None):
    """Y [T, out] bf16 = X_hat W_hat^T + (alpha/r) (X A^T) B^T, X_hat = X
    quantized per row and 128 columns; r = 0: no adapter (A, B None)."""
    T, _ = _matrix(X, "X")
    dev = X.device
    _arg(X, torch.bfloat16, (T, W.cols), "X", dev)
    _fp8_args(W, A, B, r, dev)
    if Y is None:
        Y = torch.empty(T, W.rows, dtype=torch.bfloat16, device=dev)
    else:
        _rows_arg(Y, torch.bfloat16, T, W.rows, "Y", dev)
    ws = _scratch(ws, qlora_fp8_workspace_bytes(T, W.cols, W.rows, r, False), dev)
    _on(dev, _lib.qlora_fp8_linear_fwd, "qlora_fp8_linear_fwd", ctypes.byref(W._c()), X.data_ptr(), T,
        A.data_ptr() if r > 0 else None, B.data_ptr() if r > 0 else None, r, float(alpha), Y.data_ptr(),
        ws.data_ptr(), ws.numel() * ws.element_size())
    return Y


def qlora_fp8_linear_bwd(W: FP8Weight, X, dY, A, B, r: int, alpha: float, dX=None, dA=None, dB=None, ws=None):
    """-> (dX [T, in] bf16, dA [r, in] fp32, dB [out, r] fp32); r = 0: (dX,
    None, None), and X, A, B may be None."""
    T, _ = _matrix(dY, "dY")
    dev = dY.device
    _arg(dY, torch.bfloat16, (T, W.rows), "dY", dev)
    if r > 0:
        _arg(X, torch.bfloat16, (T, W.cols), "X", dev)
    _fp8_args(W, A, B, r, dev)
    if dX is None:
        dX = torch.empty(T, W.cols, dtype=torch.bfloat16, device=dev)
    else:
        _rows_arg(dX, torch.bfloat16, T, W.cols, "dX", dev)
    if r > 0:
        if dA is None:
            dA = torch.empty(r, W.cols, dtype=torch.float32, device=dev)
        else:
            _rows_arg(dA, torch.float32, r, W.cols, "dA", dev)
        if dB is None:
            dB = torch.empty(W.rows, r, dtype=torch.float32, device=dev)
        else:
            _rows_arg(dB, torch.float32, W.rows, r, "dB", dev)
    else:
        X = A = B = dA = dB = None
    ws = _scratch(ws, qlora_fp8_workspace_bytes(T, W.cols, W.rows, r, True), dev)
    ptr = (lambda t: t.data_ptr() if t is not None else None)
    _on(dev, _lib.qlora_fp8_linear_bwd, "qlora_fp8_linear_bwd", ctypes.byref(W._c()), ptr(X), dY.data_ptr(), T,
        ptr(A), ptr(B), r, float(alpha), dX.data_ptr(), ptr(dA), ptr(dB), ws.data_ptr(),
        ws.numel() * ws.element_size())
    return dX, dA, dB


def qlora_moe_route(logits, k: int, renormalize: bool = True, ids=None, weights=None):
    """fp32 logits [T, E] -> (ids int32 [T, k], weights fp32 [T, k]): the k
    largest (ties to the lower index) and their softmax weights, over the k
    chosen (renormalize) or over all E."""
    T, E = _matrix(logits, "logits")
    dev = logits.device
    _arg(logits, torch.float32, T * E, "logits", dev)
    if ids is None:
        ids = torch.empty(T, max(k, 0), dtype=torch.int32, device=dev)
    else:
        _rows_arg(ids, torch.int32, T, k, "ids", dev)
    if weights is None:
        weights = torch.empty(T, max(k, 0), dtype=torch.float32, device=dev)
    else:
        _rows_arg(weights, torch.float32, T, k, "weights", dev)
    _on(dev, _lib.qlora_moe_route, "qlora_moe_route", logits.data_ptr(), T, E, k, 1 if renormalize else 0,
        ids.data_ptr(), weights.data_ptr())
    return ids, weights


def qlora_moe_route_bwd(logits, ids, dweights, renormalize: bool = True, dlogits=None):
    """-> dlogits fp32 [T, E] for the gradient dweights [T, k] of the weights."""
    T, E = _matrix(logits, "logits")
    _, k = _matrix(ids, "ids")
    dev = logits.device
    _arg(logits, torch.float32, T * E, "logits", dev)
    _arg(ids, torch.int32, (T, k), "ids", dev)
    _arg(dweights, torch.float32, (T, k), "dweights", dev)
    if dlogits is None:
        dlogits = torch.empty(T, E, dtype=torch.float32, device=dev)
    else:
        _rows_arg(dlogits, torch.float32, T, E, "dlogits", dev)
    _on(dev, _lib.qlora_moe_route_bwd, "qlora_moe_route_bwd", logits.data_ptr(), ids.data_ptr(),
        dweights.data_ptr(), T, E, k, 1 if renormalize else 0, dlogits.data_ptr())
    return dlogits


@functools.lru_cache(maxsize=4096)
def qlora_moe_workspace_bytes(T: int, hidden: int, inter: int, k: int) -> int:
    return int(_lib.qlora_moe_workspace_bytes(T, hidden, inter, k))


def _nf4_arg(W, name, dev):
    n = W.rows * W.cols
    _arg(W.codes, torch.uint8, n // 2, name + ".codes", dev)
    if W.flags == 0:
        _arg(W.absmax_q, torch.uint8, n // 64, name + ".absmax_q", dev)
        _arg(W.absmax_scale, torch.float32, -(-n // 16384), name + ".absmax_scale", dev)


def qlora_moe_fwd(gate_up: NF4Weight, down: NF4Weight, experts: int, X, ids, weights, Y=None, ws=None):
    """Y [T, hidden] bf16: the expert layer for up to 64 tokens, Y_t = sum_j
    weights[t, j] Wd_e (silu(Wg_e x_t) * (Wu_e x_t)), e = ids[t, j].  gate_up
    [experts * 2 * inter, hidden] (an expert's gate rows, then its up rows),
    down [experts * hidden, inter]; an id outside [0, experts) adds nothing."""
    T, _ = _matrix(X, "X")
    _, k = _matrix(ids, "ids")
    dev = X.device
    hidden, inter = gate_up.cols, down.cols
    _arg(X, torch.bfloat16, (T, hidden), "X", dev)
    _arg(ids, torch.int32, (T, k), "ids", dev)
    _arg(weights, torch.float32, (T, k), "weights", dev)
    _nf4_arg(gate_up, "gate_up", dev)
    _nf4_arg(down, "down", dev)
    if Y is None:
        Y = torch.empty(T, hidden, dtype=torch.bfloat16, device=dev)
    else:
        _rows_arg(Y, torch.bfloat16, T, hidden, "Y", dev)
    ws = _scratch(ws, qlora_moe_workspace_bytes(T, hidden, inter, k), dev)
    _on(dev, _lib.qlora_moe_fwd, "qlora_moe_fwd", ctypes.byref(gate_up._c()), ctypes.byref(down._c()), experts,
        X.data_ptr(), T, ids.data_ptr(), weights.data_ptr(), k, Y.data_ptr(), ws.data_ptr(),
        ws.numel() * ws.element_size())
    return Y


# ---------------------------------------------------------------------------
# Around the layers of a training step: norm, loss through the output head,
# optimizer.  As above, a call runs on its tensors' GPU and that GPU's current
# stream.
# ---------------------------------------------------------------------------
@dataclass
class FP8Rows:
    """Quantized rows of a matrix [T, cols]: e4m3 codes, padded with 0 to whole
    blocks of 128 columns, and scale bytes by groups of four blocks (block b of
    row t: scales[b // 4, t, b % 4])."""
    codes: torch.Tensor   # uint8 [T, cols rounded up to 128]
    scales: torch.Tensor  # uint8 [ceil(cols/512), T rounded up to 256, 4]
    T: int
    cols: int


def qlora_fp8_rows_bytes(T: int, cols: int):
    c, s = _sz(), _sz()
    _check(_lib.qlora_fp8_rows_bytes(T, cols, ctypes.byref(c), ctypes.byref(s)), "qlora_fp8_rows_bytes")
    return c.value, s.value


def _rows8_arg(rows, T: int, cols: int, dev):
    if not isinstance(rows, FP8Rows):
        raise TypeError(f"rows: expected FP8Rows, got {type(rows).__name__}")
    if rows.T != T or rows.cols != cols:
        raise ValueError(f"rows: expected [{T}, {cols}], got [{rows.T}, {rows.cols}]")
    _arg(rows.codes, torch.uint8, (T, -(-cols // 128) * 128), "rows.codes", dev)
    _arg(rows.scales, torch.uint8, (-(-cols // 512), -(-T // 256) * 256, 4), "rows.scales", dev)


def qlora_fp8_linear_fwd_rows(W: FP8Weight, rows: FP8Rows, X, A, B, r: int, alpha: float, Y=None, ws=None):
    """qlora_fp8_linear_fwd of an X whose quantized rows are at hand (the same
    Y bit for bit); X None: r = 0, and more than 16 tokens or 8192 columns."""
    if not isinstance(rows, FP8Rows):
        raise TypeError(f"rows: expected FP8Rows, got {type(rows).__name__}")
    T, dev = rows.T, rows.codes.device
    _rows8_arg(rows, T, W.cols, dev)
    if X is not None:
        _arg(X, torch.bfloat16, (T, W.cols), "X", dev)
    _fp8_args(W, A, B, r, dev)
    if Y is None:
        Y = torch.empty(T, W.rows, dtype=torch.bfloat16, device=dev)
    else:
        _rows_arg(Y, torch.bfloat16, T, W.rows, "Y", dev)
    ws = _scratch(ws, qlora_fp8_workspace_bytes(T, W.cols, W.rows, r, False), dev)
    _on(dev, _lib.qlora_fp8_linear_fwd_rows, "qlora_fp8_linear_fwd_rows", ctypes.byref(W._c()), rows.codes.data_ptr(),
        rows.scales.data_ptr(), X.data_ptr() if X is not None else None, T, A.data_ptr() if r > 0 else None,
        B.data_ptr() if r > 0 else None, r, float(alpha), Y.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return Y


def qlora_rmsnorm_fwd(x, weight, residual=None, eps: float = 1e-6, y16: bool = True, rows8: bool = False, h=None, y=None,
                      rows=None, rstd=None):
    """-> (y bf16 [T, H] or None, FP8Rows of y or None, h bf16 [T, H], rstd fp32
    [T]): h = bf16(x + residual) (x itself without one), rstd = 1 / sqrt(mean
    h^2 + eps), y = bf16(h rstd weight), weight fp32 [H].  y16, rows8: which
    forms of y are wanted (up to 16 rows and 8192 columns the 8-bit layer reads y16
    alone).  h may be x or residual."""
    T, H = _matrix(x, "x")
    dev = x.device
    _arg(x, torch.bfloat16, (T, H), "x", dev)
    _arg(weight, torch.float32, H, "weight", dev)
    if residual is not None:
        _arg(residual, torch.bfloat16, (T, H), "residual", dev)
        if h is None:
            h = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        else:
            _rows_arg(h, torch.bfloat16, T, H, "h", dev)
    elif h is not None and h is not x:
        raise ValueError("h: is x without a residual")
    y16, rows8 = y16 or y is not None, rows8 or rows is not None
    if not y16 and not rows8:
        raise ValueError("y16, rows8: one of them is needed")
    if y is not None:
        _rows_arg(y, torch.bfloat16, T, H, "y", dev)
    elif y16:
        y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    if rows is not None:
        _rows8_arg(rows, T, H, dev)
    elif rows8:
        rows = FP8Rows(torch.empty(T, -(-H // 128) * 128, dtype=torch.uint8, device=dev),
                       torch.empty(-(-H // 512), -(-T // 256) * 256, 4, dtype=torch.uint8, device=dev), T, H)
    if rstd is None:
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
    else:
        _arg(rstd, torch.float32, T, "rstd", dev)
    _on(dev, _lib.qlora_rmsnorm_fwd, "qlora_rmsnorm_fwd", x.data_ptr(), residual.data_ptr() if residual is not None else None,
        weight.data_ptr(), T, H, float(eps), h.data_ptr() if residual is not None else None,
        y.data_ptr() if y is not None else None, rows.codes.data_ptr() if rows8 else None,
        rows.scales.data_ptr() if rows8 else None, rstd.data_ptr())
    return y, rows, x if residual is None else h, rstd


@functools.lru_cache(maxsize=4096)
def qlora_rmsnorm_workspace_bytes(T: int, H: int) -> int:
    return int(_lib.qlora_rmsnorm_workspace_bytes(T, H))


def qlora_rmsnorm_bwd(dy, h, weight, rstd, dres=None, want_dweight: bool = True, dh=None, dweight=None, ws=None):
    """-> (dh bf16 [T, H], dweight fp32 [H] or None), h and rstd as the forward
    gave them; dres: the gradient that reaches h past the norm.  dh may be dy or
    dres."""
    T, H = _matrix(dy, "dy")
    dev = dy.device
    _arg(dy, torch.bfloat16, (T, H), "dy", dev)
    _arg(h, torch.bfloat16, (T, H), "h", dev)
    _arg(weight, torch.float32, H, "weight", dev)
    _arg(rstd, torch.float32, T, "rstd", dev)
    if dres is not None:
        _arg(dres, torch.bfloat16, (T, H), "dres", dev)
    if dh is None:
        dh = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    else:
        _rows_arg(dh, torch.bfloat16, T, H, "dh", dev)
    ws_ptr, ws_bytes = None, 0
    if dweight is not None:
        _arg(dweight, torch.float32, H, "dweight", dev)
    elif want_dweight:
        dweight = torch.empty(H, dtype=torch.float32, device=dev)
    if dweight is not None:
        ws = _scratch(ws, qlora_rmsnorm_workspace_bytes(T, H), dev)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _on(dev, _lib.qlora_rmsnorm_bwd, "qlora_rmsnorm_bwd", dy.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
        dres.data_ptr() if dres is not None else None, T, H, dh.data_ptr(),
        dweight.data_ptr() if dweight is not None else None, ws_ptr, ws_bytes)
    return dh, dweight


@functools.lru_cache(maxsize=4096)
def qlora_head_workspace_bytes(T: int, vocab: int, hidden: int, expand: bool, grad: bool) -> int:
    return int(_lib.qlora_head_workspace_bytes(T, vocab, hidden, 1 if expand else 0, 1 if grad else 0))


def _head_args(W, X, labels, grad: bool, loss, lse, ws):
    """Checks what both calls take -> (T, H, the head's C struct, loss, lse, workspace)."""
    T, H = _matrix(X, "X")
    dev = X.device
    _arg(X, torch.bfloat16, (T, H), "X", dev)
    head = _HeadC(hidden=H)
    if isinstance(W, NF4Weight):
        vocab = W.rows
        if W.flags == QLORA_NF4_ABSMAX_FP32:
            _arg(W.codes, torch.uint8, vocab * W.cols // 2, "W.codes", dev)
            _arg(W.absmax_scale, torch.float32, vocab * W.cols // 64, "W.absmax_scale", dev)
        else:
            _nf4_arg(W, "W", dev)
        head.nf4 = ctypes.pointer(W._c())
    elif isinstance(W, FP8Weight):
        vocab = W.rows
        _fp8_args(W, None, None, 0, dev)
        head.fp8 = ctypes.pointer(W._c())
    else:
        vocab, _ = _matrix(W, "W")
        _arg(W, torch.bfloat16, (vocab, H), "W", dev)
        head.bf16 = W.data_ptr()
    head.vocab = vocab
    _arg(labels, torch.int64, T, "labels", dev)
    if loss is None:
        loss = torch.empty(T, dtype=torch.float32, device=dev)
    else:
        _arg(loss, torch.float32, T, "loss", dev)
    if lse is None:
        lse = torch.empty(T, dtype=torch.float32, device=dev)
    else:
        _arg(lse, torch.float32, T, "lse", dev)
    ws = _scratch(ws, qlora_head_workspace_bytes(T, vocab, H, not head.bf16, grad), dev)
    return T, H, head, loss, lse, ws


def qlora_head_loss(W, X, labels, loss=None, lse=None, ws=None):
    """-> (loss fp32 [T], lse fp32 [T]) of the logits X W^T: loss = lse -
    logit[label], 0 where the label is outside [0, vocab).  W: the frozen output
    head [vocab, hidden], a bf16 tensor, an NF4Weight or an FP8Weight; X bf16 [T,
    hidden]; labels int64 [T]."""
    T, _, head, loss, lse, ws = _head_args(W, X, labels, False, loss, lse, ws)
    _on(X.device, _lib.qlora_head_loss, "qlora_head_loss", ctypes.byref(head), X.data_ptr(), T, labels.data_ptr(),
        loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return loss, lse


def qlora_head_loss_grad(W, X, labels, dloss, loss=None, lse=None, dX=None, ws=None):
    """-> (loss, lse, dX bf16 [T, hidden]): qlora_head_loss and the gradient of X
    for dloss fp32 [T], the gradient of each row's loss; the logits are formed
    once for both."""
    T, H, head, loss, lse, ws = _head_args(W, X, labels, True, loss, lse, ws)
    dev = X.device
    _arg(dloss, torch.float32, T, "dloss", dev)
    if dX is None:
        dX = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    else:
        _rows_arg(dX, torch.bfloat16, T, H, "dX", dev)
    _on(dev, _lib.qlora_head_loss_grad, "qlora_head_loss_grad", ctypes.byref(head), X.data_ptr(), T, labels.data_ptr(),
        dloss.data_ptr(), loss.data_ptr(), lse.data_ptr(), dX.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return loss, lse, dX


@dataclass
class AdamWState:
    """The states of all tensors of a plan, one tensor's after another's, each
    rounded up to 128 elements.  32 bits: m, v fp32.  8 bits: m, v uint8 (e4m3
    codes of m and of sqrt(v)) with scale bytes, one per 128 elements."""
    m: torch.Tensor
    v: torch.Tensor
    m_scales: torch.Tensor = None
    v_scales: torch.Tensor = None


@dataclass
class AdamWPlan:
    """Tensors bound to an optimizer's step.  It keeps them (their memory is
    read and written at every step; a tensor whose storage is replaced needs a new
    plan).  A graph that holds its steps needs it for as long as it is replayed."""
    state: AdamWState
    bits: int
    offsets: list     # each tensor's first element in the states
    tensors: list     # what the table points to
    table: torch.Tensor
    _c: _AdamWTableC
    _stream: int = 0  # the table was allocated on


def _numels(numel):
    return (_i64 * max(len(numel), 1))(*[int(n) for n in numel])


def qlora_adamw_state_len(numel) -> int:
    """Elements of m and of v for tensors of these sizes."""
    n = int(_lib.qlora_adamw_state_len(_numels(numel), len(numel)))
    if n < 0:
        raise QloraError(-2, "qlora_adamw_state_len")
    return n


def qlora_adamw_state(numel, bits: int, device) -> AdamWState:
    """Zero states for tensors of these sizes."""
    if bits not in (8, 32):
        raise ValueError(f"bits: 8 or 32, got {bits}")
    n = qlora_adamw_state_len(numel)
    if bits == 32:
        return AdamWState(torch.zeros(n, dtype=torch.float32, device=device),
                          torch.zeros(n, dtype=torch.float32, device=device))
    return AdamWState(*[torch.zeros(k, dtype=torch.uint8, device=device) for k in (n, n, n // 128, n // 128)])


def qlora_adamw_plan(params, masters, grads, state: AdamWState) -> AdamWPlan:
    """Binds tensors to their states.  params: bf16 tensors or None, masters: fp32
    tensors or None (one of the two per tensor, or both: the master and the copy
    that the layers read; either list may be None), grads: fp32, of the same sizes.
    The dA, dB of the layers are written into grads with their output arguments.
    Waits for the current stream; not while it is being captured."""
    n = len(grads)
    params, masters = params if params is not None else [None] * n, masters if masters is not None else [None] * n
    if len(params) != n or len(masters) != n:
        raise ValueError(f"params, masters, grads: {len(params)}, {len(masters)} and {n} tensors")
    if not isinstance(state, AdamWState) or not isinstance(state.m, torch.Tensor):
        raise TypeError(f"state: expected an AdamWState, got {type(state).__name__}")
    dev = state.m.device
    bits = 8 if state.m.dtype == torch.uint8 else 32
    numel, offsets, total = [], [], 0
    for i, (p, f, g) in enumerate(zip(params, masters, grads)):
        if not isinstance(g, torch.Tensor):
            raise TypeError(f"grads[{i}]: expected a tensor, got {type(g).__name__}")
        if p is None and f is None:
            raise TypeError(f"params[{i}], masters[{i}]: one of them is needed")
        shape, k = g.shape, g.numel()
        _arg(g, torch.float32, shape, "grads", dev, i)
        if p is not None:
            _arg(p, torch.bfloat16, shape, "params", dev, i)
        if f is not None:
            _arg(f, torch.float32, shape, "masters", dev, i)
        numel.append(k)
        offsets.append(total)
        total += -(-k // 128) * 128
    length = qlora_adamw_state_len(numel)
    kind = torch.uint8 if bits == 8 else torch.float32
    _arg(state.m, kind, length, "state.m", dev)
    _arg(state.v, kind, length, "state.v", dev)
    if bits == 8:
        _arg(state.m_scales, torch.uint8, length // 128, "state.m_scales", dev)
        _arg(state.v_scales, torch.uint8, length // 128, "state.v_scales", dev)
    if _capturing(dev):
        raise RuntimeError("qlora_adamw_plan: the current stream is being captured")
    need = int(_lib.qlora_adamw_table_bytes(_numels(numel), n))
    table = torch.empty(need, dtype=torch.uint8, device=dev)
    ptr = (lambda t: t.data_ptr() if t is not None else None)
    rows = (_AdamWTensorC * max(n, 1))(*[_AdamWTensorC(ptr(p), ptr(f), g.data_ptr(), k)
                                         for p, f, g, k in zip(params, masters, grads, numel)])
    out = _AdamWTableC()
    _on(dev, _lib.qlora_adamw_plan, "qlora_adamw_plan", rows, n, table.data_ptr(), need, ctypes.byref(out))
    # aliases of the tensors: what they point to stays allocated
    kept = [t.detach() for ts in (params, masters, grads) for t in ts if t is not None]
    return AdamWPlan(AdamWState(*[t.detach() if t is not None else None for t in
                                  (state.m, state.v, state.m_scales, state.v_scales)]), bits, offsets, kept, table, out,
                     _raw_stream(dev.index))


def qlora_adamw_step(plan: AdamWPlan, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                     weight_decay: float = 0.0, grad_scale=None, seed: int = None):
    """One AdamW step (the step-th, from 1 on) over all tensors of a plan, in
    place.  grad_scale: fp32 tensor of one element on the GPU, multiplied into every
    gradient; seed: of the 8-bit states' rounding (the step's number if None)."""
    st = plan.state
    dev = plan.table.device
    if grad_scale is not None:
        _arg(grad_scale, torch.float32, 1, "grad_scale", dev)
    small = plan.bits == 8
    # a table that went back to the allocator under a step would lead it anywhere
    if _raw_stream(dev.index) != plan._stream and not _capturing(dev):
        plan.table.record_stream(torch.cuda.current_stream(dev))
    rates = _AdamWRatesC(lr, beta1, beta2, eps, weight_decay, step, (step if seed is None else seed) & 0xffffffff)
    _on(dev, _lib.qlora_adamw_step, "qlora_adamw_step", ctypes.byref(plan._c), plan.bits, st.m.data_ptr(), st.v.data_ptr(),
        st.m_scales.data_ptr() if small else None, st.v_scales.data_ptr() if small else None,
        grad_scale.data_ptr() if grad_scale is not None else None, ctypes.byref(rates))
