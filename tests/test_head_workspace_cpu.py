"""The head loss's workspace against the largest sizes that the header names."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.environ.get("QLORA_ABI_LIB") or os.path.join(ROOT, "bit_nf4_quantized_20_amd", "libqlora.so")

TOKENS = (1, 16, 32, 33, 64, 65, 128, 129, 256, 300, 511, 512, 513, 600, 1000, 1024, 2047, 2048, 2304, 2500, 3500, 4095, 4096, 4097, 6000,
          8192, 8193, 12289, 1 << 20, (1 << 31) - 1)
VOCABS = (1, 63, 64, 1000, 4160, 8256, 16384, 32000, 32768, 50021, 65536, 100000, 128000, 128256, 131072, 200000, 262144, 1 << 19, 1 << 20,
          1 << 21, 1 << 22, 1 << 23, (1 << 24) - 64, 1 << 24)
HIDDEN = (64, 128, 192, 320, 1024, 2048, 2304, 4096, 4160, 8192, 12288, 16320, 16384)


@pytest.mark.parametrize("expand,grad,most", [(0, 0, 521), (0, 1, 521), (1, 1, 585), (1, 0, 769)])
def test_workspace_stays_within_what_the_header_says(expand, grad, most):
    lib = ctypes.CDLL(LIB)
    size = lib.qlora_head_workspace_bytes
    size.restype, size.argtypes = ctypes.c_size_t, [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    for T in TOKENS:
        for V in VOCABS:
            if expand and V % 64:
                continue
            for H in HIDDEN:
                assert 0 < size(T, V, H, expand, grad) <= most << 20, (T, V, H)
    header = open(os.path.join(ROOT, "include", "qlora.h")).read()
    assert f"{most}" in header
