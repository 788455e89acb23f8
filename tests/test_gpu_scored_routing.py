"""Routing by scores and its gradient against the float64 oracle.

Tolerances.  Picks are whole numbers and equal.  Weights are computed in 64 bits and
rounded once: half a step, 2^-24 of the value (and 1e-12 for the 64-bit part).  The
gradient's parts are computed in 64 bits and rounded to fp32, 2^-24, and so is an
addition to what is there or of an id that a row holds twice; softmax scores that are
not renormalised take up to 6 more roundings of their terms: 8 2^-24 of the sum of
the terms' magnitudes in all."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import scored_routing as sr

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def _dev(a, stride=None, offset=0, fill=float("nan")):
    """a's rows on the device, `stride` elements apart, the first at an offset of `offset` elements."""
    if stride is None and not offset:
        return torch.from_numpy(np.ascontiguousarray(a)).to(gh.dev())
    R, C = a.shape
    flat = torch.full((offset + R * (stride or C),), fill, dtype=torch.float32, device=gh.dev())
    v = flat[offset:].view(R, stride or C)
    v[:, :C] = torch.from_numpy(a).to(gh.dev())
    return v


def _route(z, k, kind, bias=None, groups=1, kept=1, top=1, renorm=True, scale=1.0, stride=None, offset=0):
    T, E = z.shape
    r = lib.make_router(E, k, kind, groups, kept, top, renorm, scale)
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device=gh.dev())
    w = torch.full((T + 1, k), 7.0, device=gh.dev())
    b = None if bias is None else torch.from_numpy(bias).to(gh.dev())
    lib.moe_route_scores(r, T, _dev(z, stride, offset), ids, w, bias=b, logits_stride=stride)
    torch.cuda.synchronize()
    assert (ids[T] == -7).all() and (w[T] == 7).all()  # rows behind the last token
    return ids[:T].cpu().numpy(), w[:T].cpu().numpy()


def _check(z, k, kind, *a, stride=None, offset=0):
    ids, w = _route(z, k, kind, *a, stride=stride, offset=offset)
    rid, rw = sr.route(z, k, kind, *a)
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:5]
    assert (np.abs(w - rw) <= EPS * (1 + 1e-4) * np.abs(rw) + 1e-45).all()


GROUPS = [(1, 1, 1), (8, 4, 2), (4, 1, 1), (4, 3, 2), (16, 5, 2), (2, 1, 2)]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [1, 3, 16, 48, 64, 65, 96, 160, 255, 256, 257, 384, 512, 1000, 1024])
def test_experts(kind, E):
    rng = np.random.default_rng(E)
    for T in (1, 5, 67):
        z = (2 * rng.standard_normal((T, E))).astype(np.float32)
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        for i, (G, KG, top) in enumerate(GROUPS):
            if E % G or top > E // G:
                continue
            k = min(KG * (E // G), (8, 6, 1, 10, 17, 32)[i])
            _check(z, k, kind, bias if i % 2 == 0 else None, G, KG, top, i % 3 != 1, 2.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,KG,k", [(256, 8, 4, 8), (160, 8, 3, 6), (60, 6, 2, 4), (64, 1, 1, 16), (100, 50, 9, 16),
                                      (7, 1, 1, 7), (256, 128, 30, 12)])
def test_many_tokens(kind, E, G, KG, k):
    rng = np.random.default_rng(E + k)
    z = (2 * rng.standard_normal((2050, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    _check(z, k, kind, bias, G, KG, 2 if E // G > 1 else 1, True, 0.75)
    _check(z, k, kind, None, G, KG, 1, False, 1.0, stride=E + 3, offset=1)


@pytest.mark.parametrize("stride,offset", [(256, 0), (257, 0), (260, 0), (256, 1), (264, 2), (512, 4)])
@pytest.mark.parametrize("T", [9, 2100])
def test_strides_and_alignment(stride, offset, T):
    z = np.random.default_rng(3).standard_normal((T, 256)).astype(np.float32)
    _check(z, 8, "sigmoid", None, 8, 4, 2, True, 1.0, stride=stride, offset=offset)


@pytest.mark.parametrize("T", [40, 2100])
def test_equal_choices(T):
    """Logits of few values, and saturated scores: equal choices go to the lower id, equal groups to the lower group."""
    rng = np.random.default_rng(4)
    z = rng.integers(-2, 3, (T, 64)).astype(np.float32)
    z[1::4] = 0.0
    z[2::4] = -0.0
    z[3::4] += 40.0  # sigmoid is 1 in 32 bits
    for kind in ("softmax", "sigmoid"):
        _check(z, 8, kind, None, 8, 3, 2, True, 1.0)
        _check(z, 8, kind, np.zeros(64, np.float32), 1, 1, 1, False, 1.0)


@pytest.mark.parametrize("T", [40, 2100])
def test_experts_that_are_switched_off(T):
    """Rows with one expert left, with fewer than k, with none: picks are in range and different, weights of experts that
    are off 0, and 0 where all of a row's are."""
    rng = np.random.default_rng(5)
    z = rng.standard_normal((T, 128)).astype(np.float32)
    z[:, 5] = z[:, 77] = -np.inf
    z[1::5, :] = -np.inf
    z[2::5, 1:] = -np.inf
    z[3::5, 4:] = -np.inf
    bias = rng.standard_normal(128).astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        for groups in ((1, 1, 1), (8, 4, 2), (8, 4, 1)):
            _check(z, 6, kind, bias, *groups, True, 1.5)
            _check(z, 6, kind, None, *groups, False, 1.5)


@pytest.mark.parametrize("T", [30, 2100])
def test_logits_at_the_ends_of_the_type(T):
    z = np.random.default_rng(6).standard_normal((T, 96)).astype(np.float32)
    top, low = np.finfo(np.float32).max, np.finfo(np.float32).min
    z[1::7], z[2::7], z[3::7, ::2], z[4::7, ::3], z[5::7] = low, top, low, top, z[5::7] * 300
    for kind in ("softmax", "sigmoid"):
        _check(z, 7, kind, None, 4, 2, 2, True, 1.0)
        _check(z, 7, kind, None, 1, 1, 1, False, 1.0)


@pytest.mark.parametrize("T", [30, 2100])
def test_rows_that_are_not_finite(T):
    """Other rows are what they were; ids stay in range and differ."""
    z = np.random.default_rng(7).standard_normal((T, 64)).astype(np.float32)
    ids0, w0 = _route(z, 6, "softmax", None, 8, 4, 2)
    bad = np.arange(T) % 5 == 2
    z[bad, 3] = np.nan
    z[1::10, 9] = np.inf
    bad[1::10] = True
    ids, w = _route(z, 6, "softmax", None, 8, 4, 2)
    assert np.array_equal(ids[~bad], ids0[~bad]) and np.array_equal(w[~bad], w0[~bad])
    assert np.isnan(w[bad]).any(axis=1).all()
    assert ((ids >= 0) & (ids < 64)).all() and all(len(set(r)) == 6 for r in ids.tolist())
    ids, w = _route(z, 6, "sigmoid", np.full(64, np.nan, np.float32))
    assert ((ids >= 0) & (ids < 64)).all() and all(len(set(r)) == 6 for r in ids.tolist())


# ------------------------------------------------------------------ gradient


def _grad(z, ids, dw, kind, renorm, scale, mask=None, start=None, stride=None, dstride=None, offset=0):
    T, E = z.shape
    d = gh.dev()
    r = lib.make_router(E, ids.shape[1], kind, renormalise=renorm, scale=scale)
    out = _dev(np.zeros((T + 1, E), np.float32) if start is None else np.vstack([start, start[:1]]), dstride or E, offset,
               fill=3.0)
    out[T] = 5.0
    m = None if mask is None else torch.from_numpy(mask).to(d)
    lib.moe_route_scores_backward(r, T, _dev(z, stride, offset), torch.from_numpy(ids).to(d),
                                  torch.from_numpy(dw).to(d), out, token_mask=m, accumulate=start is not None,
                                  logits_stride=stride, d_logits_stride=dstride)
    torch.cuda.synchronize()
    assert (out[T] == 5.0).all() and (out[:T, E:] == 3.0).all()
    return out[:T, :E].cpu().numpy()


def _close(g, ref, mag, add=0.0):
    bad = np.abs(g - ref) > 8 * EPS * (mag + np.abs(add)) + 1e-44
    assert not bad.any(), (np.argwhere(bad)[:5], g[bad][:5], ref[bad][:5])


def _case(T, E, k, seed):
    rng = np.random.default_rng(seed)
    z = (2 * rng.standard_normal((T, E))).astype(np.float32)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, z, ids, rng.standard_normal((T, k)).astype(np.float32)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 2), (33, 64, 6), (7, 255, 8), (65, 256, 8), (5, 1000, 32),
                                   (2049, 96, 10), (2051, 256, 16), (2060, 30, 3), (2060, 64, 20)])
def test_gradient(kind, renorm, T, E, k):
    rng, z, ids, dw = _case(T, E, k, T + E)
    _close(_grad(z, ids, dw, kind, renorm, 2.5), *sr.backward(z, ids, dw, kind, renorm, 2.5))
    mask = (rng.random(T) < 0.6).astype(np.uint8)
    start = rng.standard_normal((T, E)).astype(np.float32)
    ref, mag = sr.backward(z, ids, dw, kind, renorm, 2.5, mask)
    g = _grad(z, ids, dw, kind, renorm, 2.5, mask, start, stride=E + 1, dstride=E + 2, offset=1)
    _close(g, ref + start, mag, start)
    assert np.array_equal(g[mask == 0], start[mask == 0])
    g = _grad(z, ids, dw, kind, renorm, 2.5, mask, dstride=(E + 7) // 4 * 4)
    _close(g, ref, mag)
    assert not g[mask == 0].any()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [12, 2100])
def test_gradient_of_odd_picks(kind, renorm, T):
    """Ids outside [0, E), an id twice in a row, and masked rows with anything in them."""
    rng, z, ids, dw = _case(T, 64, 4, 9)
    ids[::3, 1] = ids[::3, 0]
    ids[1::3, 2] = 64
    ids[2::6, 3] = -1
    ids[5::12] = 1 << 30
    mask = (np.arange(T) % 7 != 3).astype(np.uint8)
    ref, mag = sr.backward(z, ids, dw, kind, renorm, 1.0, mask)
    gone = mask == 0
    z[gone], dw[gone], ids[gone] = np.nan, np.inf, -(1 << 30)
    _close(_grad(z, ids, dw, kind, renorm, 1.0, mask), ref, mag)


@pytest.mark.parametrize("T,stride", [(50, 64), (2100, 64), (50, 65)])
def test_masked_rows_stay_as_they_are(T, stride):
    """Adding to what is there leaves a masked row's bits alone: negative zeros and NaN too."""
    rng, z, ids, dw = _case(T, 64, 4, 13)
    mask = (np.arange(T) % 3 == 0).astype(np.uint8)
    start = np.full((T, 64), -0.0, np.float32)
    start[:, ::5], start[:, 1::5] = np.nan, -np.inf
    g = _grad(z, ids, dw, "softmax", False, 1.0, mask, start, dstride=stride)
    assert np.array_equal(g[mask == 0].view(np.uint32), start[mask == 0].view(np.uint32))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_of_switched_off_experts(kind):
    rng, z, ids, dw = _case(40, 32, 4, 10)
    z[::2, 3] = -np.inf
    z[1::4] = -np.inf
    ids[::2, 0] = 3
    for renorm in (True, False):
        _close(_grad(z, ids, dw, kind, renorm, 1.0), *sr.backward(z, ids, dw, kind, renorm, 1.0))


@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_is_the_weights_differences(kind, renorm):
    """Central differences of the weights that the library computes: half a step of an fp32 weight (at most 1) over the
    step h = 2^-6, twice, and h^2 / 6 of a third derivative below 1, over the k weights' gradients (at most 3.5 each)."""
    rng, z, ids, dw = _case(5, 10, 3, 11)
    z *= 0.5
    ids, w = _route(z, 3, kind, renorm=renorm)
    g, h = _grad(z, ids, dw, kind, renorm, 1.0), 2.0 ** -6
    for t in range(5):
        for e in range(10):
            v = []
            for sgn in (1, -1):
                m = z.copy()
                m[t, e] += sgn * h
                i, w = _route(m, 3, kind, renorm=renorm)
                pos = [i[t].tolist().index(a) if a in i[t] else None for a in ids[t]]
                if None in pos:
                    break
                v.append(float((dw[t].astype(np.float64) * w[t][pos]).sum()))
            if len(v) == 2:  # (a pick that changes hands has no difference)
                assert abs((v[0] - v[1]) / (2 * h) - g[t, e]) <= np.abs(dw[t]).sum() * (EPS / h + h * h / 6)


@pytest.mark.parametrize("T", [64, 4096])
def test_captured_and_on_another_stream(T):
    rng, z, ids, dw = _case(T, 256, 8, 12)
    d = gh.dev()
    r = lib.make_router(256, 8, "sigmoid", 8, 4, 2, True, 2.5)
    zd, dwd = torch.from_numpy(z).to(d), torch.from_numpy(dw).to(d)
    new = lambda: (torch.zeros(T, 8, dtype=torch.int32, device=d), torch.zeros(T, 8, device=d), torch.zeros(T, 256, device=d))  # noqa: E731

    def step(o):
        lib.moe_route_scores(r, T, zd, o[0], o[1])
        lib.moe_route_scores_backward(r, T, zd, o[0], dwd, o[2])

    ref, got = new(), new()
    step(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(got)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got)
    for i in range(3):
        zd.copy_(torch.from_numpy(np.roll(z, i, 0)))
        for o in got:
            o.zero_()
        graph.replay()
        step(ref)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_rows_far_apart():
    """Offsets past 2^31 values: the last rows of 2^21 of 1024 experts."""
    d, T, E = gh.dev(), (1 << 21) + 3, 1024
    z = torch.empty(T, E, device=d).normal_(generator=torch.Generator(device=d).manual_seed(1))
    r = lib.make_router(E, 4, "softmax", renormalise=False)
    ids, w = torch.empty(T, 4, dtype=torch.int32, device=d), torch.empty(T, 4, device=d)
    lib.moe_route_scores(r, T, z, ids, w)
    g = torch.empty(T, E, device=d)
    lib.moe_route_scores_backward(r, T, z, ids, w, g)
    at = np.r_[0:3, T - 40:T]
    zs, i, ww, gs = (v[at].cpu().numpy() for v in (z, ids, w, g))
    rid, rw = sr.route(zs, 4, "softmax", renorm=False)
    assert np.array_equal(i, rid) and (np.abs(ww - rw) <= EPS * (1 + 1e-4) * rw).all()
    _close(gs, *sr.backward(zs, i, ww, "softmax", False))
