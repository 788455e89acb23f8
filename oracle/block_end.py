"""The end of an expert block and its gradients (oracle; test infrastructure),
float64, with the sums of the terms' magnitudes beside the values: what roundings
are measured by.
"""
from __future__ import annotations

import numpy as np


def _f(v):
    return None if v is None else np.asarray(v, np.float64)


def weighted(y, w, shared, gate):
    """(m, sum of its terms' magnitudes), [T, H]."""
    m = mag = 0.0
    if y is not None:
        T, k = w.shape
        t = _f(w)[:, :, None] * _f(y).reshape(T, k, -1)
        m, mag = t.sum(1), np.abs(t).sum(1)
    if shared is not None:
        s = _f(shared) * (1.0 if gate is None else _f(gate)[:, None])
        m, mag = m + s, mag + np.abs(s)
    return m, mag


def _q(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def forward(y, w, shared, gate, res, post, nxt, eps, scale):
    """(r, normed or None, error of r by its magnitudes): the fp32 roundings' part of r's error is at most the third
    times 2^-24."""
    m, mag = weighted(y, w, shared, gate)
    k = 0 if y is None else w.shape[1]
    # a sum of k + 1 products, a norm's factor (40 additions of squares, whose root halves them, 4 more roundings)
    err = (k + 2) * mag
    if post is not None:
        q = _q(m, eps)
        err = q * np.abs(_f(post)) * (err + np.abs(m) * (q * np.sqrt((err * err).mean(1, keepdims=True)) + 26))
        m = m * q * _f(post)
    r = scale * m
    err = abs(scale) * (err + np.abs(m))
    if res is not None:
        r = r + _f(res)
    err = err + np.abs(r)
    n = None if nxt is None else r * _q(r, eps) * _f(nxt)
    return r, n, err


def backward(y, w, shared, gate, out, post, nxt, eps, scale, d_out, d_normed):
    """{name: (value, magnitude)} of every gradient that the inputs have."""
    o = {}
    ref = next(v for v in (d_out, d_normed) if v is not None)
    d = np.zeros(np.shape(ref)) if d_out is None else _f(d_out)
    a = np.abs(d)
    if nxt is not None:
        r, dn, g = _f(out), _f(d_normed), _f(nxt)
        q = _q(r, eps)
        c = dn * g
        o["d_next"] = ((dn * r * q).sum(0), np.abs(dn * r * q).sum(0))
        d = d + q * (c - r * q * q * (c * r).mean(1, keepdims=True))
        a = a + q * (np.abs(c) + np.abs(r) * q * q * np.abs(c * r).mean(1, keepdims=True))
    o["d_res"] = (d, a)
    d, a = scale * d, abs(scale) * a
    m, mag = weighted(y, w, shared, gate)
    if post is not None:
        q, g = _q(m, eps), _f(post)
        o["d_post"] = ((d * m * q).sum(0), (a * mag * q).sum(0))
        c, ca = d * g, a * np.abs(g)
        d = q * (c - m * q * q * (c * m).mean(1, keepdims=True))
        a = q * (ca + mag * q * q * (ca * mag).mean(1, keepdims=True))
    if y is not None:
        T, k = w.shape
        yy, ww = _f(y).reshape(T, k, -1), _f(w)[:, :, None]
        o["d_w"] = ((yy * d[:, None]).sum(2), (np.abs(yy) * a[:, None]).sum(2))
        o["d_y"] = ((ww * d[:, None]).reshape(T * k, -1), (np.abs(ww) * a[:, None]).reshape(T * k, -1))
    if shared is not None:
        s, gt = _f(shared), 1.0 if gate is None else _f(gate)[:, None]
        if gate is not None:
            o["d_gate"] = ((s * d).sum(1), (np.abs(s) * a).sum(1))
        o["d_shared"] = (gt * d, np.abs(gt) * a)
    return o
