"""Which kernels of the head loss the GPU tests reach: the rule that chooses the tiles
(csrc/head_shapes.hpp, host code) is asked for every size of their lists, so that a
change of it does not quietly leave a tile height untested."""

import os
import subprocess

import pytest

import test_gpu_head
import test_gpu_head_edges

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "bit_nf4_quantized_20_amd", "csrc", "head_shapes.hpp")
PROGRAM = f"""
#include "{HEADER}"
#include <cstdio>
int main() {{
  long T, V, H;
  int codes;
  while (std::scanf("%ld %ld %ld %d", &T, &V, &H, &codes) == 4) {{
    const auto l = qlora::logits_shape(T, V, codes);
    const auto g = qlora::grad_shape(T, H, V, codes);
    std::printf("%d %d %d %d %d\\n", l.rows, l.cols, g.tile.rows, g.tile.cols, g.splits);
  }}
}}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """f(sizes, codes) -> [((rows, cols) of the logits' tile, of dX's, splits)]; the sizes are of one piece."""
    at = tmp_path_factory.mktemp("shapes")
    src, exe = str(at / "shapes.cpp"), str(at / "shapes")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", exe, src], check=True, capture_output=True, timeout=120)

    def ask(sizes, codes):
        text = "".join(f"{t} {v} {h} {int(codes)}\n" for t, v, h in sizes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split()
        n = [int(x) for x in out]
        return [((n[i], n[i + 1]), (n[i + 2], n[i + 3]), n[i + 4]) for i in range(0, len(n), 5)]
    return ask


def _sizes(test):
    """The (T, V, H) that a test is parametrised with."""
    for mark in test.pytestmark:
        if mark.name == "parametrize" and mark.args[0] == "T,V,H":
            return list(mark.args[1])
    raise AssertionError(test)


HEIGHTS16 = (64, 96, 128, 160, 192, 224, 256)
SHAPES8 = [(32, 128), (64, 128), (128, 128)] + [(h, 256) for h in (96, 128, 160, 192, 256)]


def test_the_rule_takes_no_other_shape(shapes):
    sizes = [(t, v, h) for t in list(range(1, 513, 7)) + [600, 1000, 1500, 2304, 4096] for v in (1, 300, 5000, 32000, 131072)
             for h in (64, 1024, 4160, 16384)]
    for l, g, s in shapes(sizes, False):
        assert l == (64, 128) or l[1] == 256 and l[0] in HEIGHTS16
        assert g[1] == 256 and g[0] in HEIGHTS16 and s >= 1
    for l, g, s in shapes([x for x in sizes if x[0] <= 512], True):
        assert l in SHAPES8 and g in SHAPES8 and s >= 1


def test_16_bit_tiles_are_tested_next_to_their_borders(shapes):
    """Each height with its last row missing and as the next height's first, in more than one K-step and more
    than one column tile (of both products)."""
    logits, grads = test_gpu_head_edges.LOGITS, test_gpu_head_edges.GRADS
    assert set(logits + grads) == set(_sizes(test_gpu_head_edges.test_16_bit_head_of_each_tile))
    at = [(T, l[0]) for (T, V, H), (l, _, _) in zip(logits, shapes(logits, False)) if l[1] == 256 and H >= 128 and V > 512]
    dx = [(T, g[0]) for (T, V, H), (_, g, _) in zip(grads, shapes(grads, False)) if V >= 128 and H > 512]
    for seen in (at, dx):
        for low, high in zip((0,) + HEIGHTS16, HEIGHTS16):
            rows = [T for T, h in seen if h == high]
            assert any(T % high in (high - 1, 0) for T in rows), (high, rows)  # the tile full, or one row short of it
            assert high == 64 or low + 1 in rows, (high, rows)                 # as few rows as take it
    assert any(s > 1 for _, _, s in shapes(grads, False))
    # the logits' tile of 128 columns
    few = _sizes(test_gpu_head.test_loss_and_gradient)
    assert any(l == (64, 128) and H >= 128 and V > 256 for (_, V, H), (l, _, _) in zip(few, shapes(few, False)))


def test_tiles_of_codes_are_tested(shapes):
    sizes = [x for t in (test_gpu_head.test_quantized_heads, test_gpu_head.test_quantized_heads_of_each_tile,
                         test_gpu_head_edges.test_quantized_head_of_each_tile) for x in _sizes(t) if x[0] <= 512]
    seen = shapes(sizes, True)
    assert {l for (_, V, H), (l, _, _) in zip(sizes, seen) if H >= 128 and V > 256} == set(SHAPES8)
    assert {g for (_, V, H), (_, g, _) in zip(sizes, seen) if H >= 320 and V >= 128} == set(SHAPES8)
