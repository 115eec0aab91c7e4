"""The mixture-of-experts operators where their inputs leave the ordinary:
NaN and infinities in rows and in masked places, hidden values past bf16's
largest, workspaces with any contents."""

import numpy as np
import pytest
import torch

import synth
from oracle import moe as omoe

from gpu_util import banner, dev_f32, host, require_gpu

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
