"""The gradient of routing by scores where its terms cancel: every value is computed in
64 bits and rounded once.

Tolerance: half a step of the value, 2^-24, and half of the smallest number, 2^-150;
the 64-bit part is two exponentials, their sum and its reciprocal, each within 2.1e-14,
in up to three factors of a term: 2e-13 of the sum of the terms' magnitudes."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import scored_routing as sr

pytestmark = pytest.mark.gpu


def _grad(z, ids, dw, kind, renorm, scale=1.0, stride=None):
    T, E = z.shape
    d, ld = gh.dev(), stride or E
    r = lib.make_router(E, ids.shape[1], kind, renormalise=renorm, scale=scale)
    zd, out = torch.full((T, ld), 9.0, device=d), torch.full((T, ld), 7.0, device=d)
    zd[:, :E] = torch.from_numpy(z).to(d)
    lib.moe_route_scores_backward(r, T, zd, torch.from_numpy(ids).to(d), torch.from_numpy(dw).to(d), out,
                                  logits_stride=ld, d_logits_stride=ld)
    torch.cuda.synchronize()
    assert (out[:, E:] == 7.0).all()
    return out[:, :E].cpu().numpy().astype(np.float64)


def _check(z, ids, dw, kind, renorm, scale=1.0, stride=None):
    g = _grad(z, ids, dw, kind, renorm, scale, stride)
    ref, mag = sr.backward(z, ids, dw, kind, renorm, scale)
    bad = np.abs(g - ref) > 2.0 ** -24 * np.abs(ref) + 2e-13 * mag + 2.0 ** -150
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4])


FORMS = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]
SIZES = [(40, 4), (40, 64), (300, 255), (33, 1000), (4100, 96), (4200, 256)]


@pytest.mark.parametrize("kind,renorm", FORMS)
@pytest.mark.parametrize("T,E", SIZES)
def test_one_pick_far_above_the_rest(kind, renorm, T, E):
    """The pick's gradient is g p (1 - p) with p up to 1 - 1e-9: the difference of two nearly equal terms."""
    rng = np.random.default_rng(T + E)
    z = rng.standard_normal((T, E)).astype(np.float32)
    at = rng.integers(0, E, T)
    z[np.arange(T), at] += np.linspace(3.0, 24.0, T).astype(np.float32)
    _check(z, at[:, None].astype(np.int32), rng.standard_normal((T, 1)).astype(np.float32), kind, renorm, 2.5)


@pytest.mark.parametrize("kind,renorm", FORMS)
@pytest.mark.parametrize("T,E", SIZES)
def test_picks_that_share_the_whole(kind, renorm, T, E):
    """Two picks with nearly all of the weight between them and the same gradient."""
    rng = np.random.default_rng(T * E)
    z = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:3] for _ in range(T)]).astype(np.int32)
    z[np.arange(T), ids[:, 0]] += 12.0
    z[np.arange(T), ids[:, 1]] += 12.5
    dw = np.repeat(rng.standard_normal((T, 1)).astype(np.float32), 3, 1)
    _check(z, ids, dw, kind, renorm)
    _check(z, ids, dw, kind, renorm, 0.75, stride=E + 3)


@pytest.mark.parametrize("kind,renorm", FORMS)
@pytest.mark.parametrize("T,E,k", [(50, 64, 4), (4100, 128, 6), (30, 700, 32)])
def test_an_id_twice_with_parts_that_cancel(kind, renorm, T, E, k):
    rng = np.random.default_rng(T + k)
    z = (2 * rng.standard_normal((T, E))).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[::2, k - 1] = ids[::2, 0]
    ids[1::4, 2], ids[1::4, 1] = ids[1::4, 0], ids[1::4, 0]
    ids[3::4, 1] = E + 5
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dw[::2, k - 1] = -dw[::2, 0] * np.float32(1 + 2.0 ** -20)
    _check(z, ids, dw, kind, renorm)


@pytest.mark.parametrize("kind,renorm", FORMS)
@pytest.mark.parametrize("T,E,k", [(9, 1, 1), (65, 30, 3), (2050, 256, 8), (4300, 250, 16), (8, 1024, 32)])
def test_ordinary_rows(kind, renorm, T, E, k):
    rng = np.random.default_rng(T)
    z = (3 * rng.standard_normal((T, E))).astype(np.float32)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    _check(z, ids, rng.standard_normal((T, k)).astype(np.float32), kind, renorm, 2.5)
