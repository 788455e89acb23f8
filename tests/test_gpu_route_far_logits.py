"""Renormalised weights, and their gradient, of picks whose scores leave the 64-bit
numbers: the weights are the scores' ratios, whatever the scores' size.

Tolerances: as for other logits (weights half a step, 2^-24; the gradient one rounding
and 2e-13 of the terms' magnitudes)."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import scored_routing as sr

pytestmark = pytest.mark.gpu

FAR = [-30.0, -39.5, -40.0, -40.5, -87.0, -104.0, -650.0, -699.5, -700.5, -705.0, -709.0, -720.0, -740.0, -745.0, -760.0,
       -1.0e4, -3.0e38]


def _run(z, k, kind, bias, renorm):
    T, E = z.shape
    d = gh.dev()
    r = lib.make_router(E, k, kind, renormalise=renorm, scale=1.5)
    zd, bd = torch.from_numpy(z).to(d), torch.from_numpy(bias).to(d)
    ids, w = torch.zeros(T, k, dtype=torch.int32, device=d), torch.zeros(T, k, device=d)
    lib.moe_route_scores(r, T, zd, ids, w, bias=bd)
    dw = torch.from_numpy(np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)).to(d)
    g = torch.full((T, E), 7.0, device=d)
    lib.moe_route_scores_backward(r, T, zd, ids, dw, g)
    torch.cuda.synchronize()
    return [v.cpu().numpy() for v in (ids, w, dw, g)]


def _check(z, k, kind, bias, renorm):
    ids, w, dw, g = _run(z, k, kind, bias, renorm)
    rid, rw = sr.route(z, k, kind, bias, renorm=renorm, scale=1.5)
    assert np.array_equal(ids, rid)
    bad = np.abs(w - rw) > 2.0 ** -24 * (1 + 1e-4) * np.abs(rw) + 2.0 ** -150
    assert not bad.any(), (np.argwhere(bad)[:4], w[bad][:4], rw[bad][:4])
    ref, mag = sr.backward(z, ids, dw, kind, renorm, 1.5)
    bad = np.abs(g - ref) > 2.0 ** -24 * np.abs(ref) + 2e-13 * mag + 2.0 ** -150
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4])
    return w


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", [(64, 6), (256, 8), (600, 20)])
@pytest.mark.parametrize("copies", [1, 260])
def test_every_logit_far_below(kind, E, k, copies):
    """Rows around each of FAR: the weights add up to the scale as they do anywhere else."""
    rng = np.random.default_rng(E)
    z = np.repeat(np.float32(FAR), copies)[:, None] + rng.standard_normal((len(FAR) * copies, E)).astype(np.float32)
    bias = rng.standard_normal(E).astype(np.float32)
    w = _check(z, k, kind, bias, True)
    assert np.abs(w.astype(np.float64).sum(1) - 1.5).max() <= 1.5 * k * 2.0 ** -24
    _check(z, k, kind, bias, False)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [20, 2100])
def test_the_bias_picks_experts_far_below_the_others(kind, T):
    rng = np.random.default_rng(T)
    z = rng.standard_normal((T, 48)).astype(np.float32)
    far = np.float32(FAR)[np.arange(T) % len(FAR)]
    z[:, 30:34] += far[:, None]
    z[1::3, 33] = -np.inf
    z[2::5, 31] = 5.0
    bias = np.zeros(48, np.float32)
    bias[30:34] = 4.0
    _check(z, 4, kind, bias, True)


@pytest.mark.parametrize("T", [20, 2100])
def test_picks_that_are_off_have_no_weight(T):
    z = np.full((T, 16), -np.inf, np.float32)
    z[::2, 3] = np.float32(FAR)[np.arange(len(z[::2])) % len(FAR)]
    for kind in ("sigmoid", "softmax"):
        w = _check(z, 4, kind, np.zeros(16, np.float32), True)
        assert (w[::2].max(1) == 1.5).all() and not w[1::2].any()
