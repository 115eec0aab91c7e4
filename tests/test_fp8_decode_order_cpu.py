"""The few-token forward of an 8-bit weight copies the next chunk of the weight into an LDS
stage that it has just read.  In the machine code no such copy may be issued while a
read of LDS is still on its way: its data could land in rows that are yet to be read (a
handful of weights of the wrong tile in one output, now and then)."""

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "bit_nf4_quantized_20_amd")


def _builder():
    import importlib.util
    spec = importlib.util.spec_from_file_location("_qlora_build_order", os.path.join(PACKAGE, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _kernels(text):
    """Name -> instructions of each k_fp8_decode kernel."""
    out, name = {}, None
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        m = re.match(r"(_ZN5qlora12k_fp8_decode\w*):$", line)
        if m:
            name = m.group(1)
            out[name] = []
        elif name and line and not line.startswith("."):
            out[name].append(line)
            if line.startswith("s_endpgm"):
                name = None
    return out


def _early_copies(code):
    """Copies into LDS behind a read of LDS that no wait has covered.  Within straight code
    these operations end in order, so that a wait for n leaves at most the last n under way."""
    under_way, bad = 0, []
    for at, op in enumerate(code):
        if op.startswith("ds_"):
            under_way += 1
        elif op.startswith("s_waitcnt"):
            m = re.search(r"lgkmcnt\((\d+)\)", op)
            if m:
                under_way = min(under_way, int(m.group(1)))
        elif op.startswith("buffer_load") and op.endswith("lds") and under_way:
            bad.append((at, op))
    return bad


def test_the_check_finds_an_early_copy():
    read, copy, wait = "ds_read_b128 v[0:3], v9", "buffer_load_dwordx4 v4, s[4:7], 0 offen nt lds", "s_waitcnt lgkmcnt(%d)"
    assert _early_copies([read, read, wait % 1, copy]) and _early_copies([read, copy, wait % 0])
    assert not _early_copies([read, read, wait % 0, copy, copy]) and not _early_copies([copy, read])


def test_no_copy_into_lds_while_reads_are_under_way(tmp_path):
    b = _builder()
    out = str(tmp_path / "decode.s")
    cmd = [b.hipcc(), *b.flags(), "--offload-device-only", "-S", os.path.join(PACKAGE, "csrc", "k_fp8_decode.hip"), "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    kernels = _kernels(open(out).read())
    assert len(kernels) == 3
    for name, code in kernels.items():
        assert sum(op.endswith("lds") for op in code) >= 16 and sum(op.startswith("ds_read_b128") for op in code) >= 16, name
        assert not _early_copies(code), (name, _early_copies(code)[:3])
