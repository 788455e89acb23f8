"""Products on 8-bit integer weights (oracle; test infrastructure).

Weights: int8 codes [N, K] with one fp32 scale per channel.  Activations: bf16
rows, one fp32 scale per row: amax = max(max |x|, 2^-100), scale =
fp32(amax / 127), code = round(fp32(x * fp32(127 / amax))), ties to even.  Sums
of code products are integers; an output is fp32(fp32(sum) * scale_m) * scale_n.
"""
from __future__ import annotations

import numpy as np

from . import codecs

TINY = np.float32(2.0 ** -100)
TOP = np.float32(127)


def quantize_rows(v):
    """(codes int8 [R, K], scales fp32 [R]) of finite fp32 rows."""
    v = np.asarray(v, np.float32)
    amax = np.maximum(np.abs(v).max(axis=1), TINY).astype(np.float32)
    return np.rint(v * (TOP / amax)[:, None]).astype(np.int8), amax / TOP


def sums(cx, cw):
    """Integer sums [M, N]; float64 products are exact far beyond 2^31."""
    return np.rint(cx.astype(np.float64) @ cw.astype(np.float64).T).astype(np.int64)


def linear32(x_bits, codes, scales):
    """fp32 outputs [M, N] before their rounding to bf16 (three fp32 roundings, as the definition has them)."""
    cx, sx = quantize_rows(codecs.bf16_decode(x_bits))
    a = sums(cx, codes).astype(np.float32)
    return (a * sx[:, None]) * np.asarray(scales, np.float32)[None, :]


def experts(x_bits, w13, s13, w2, s2, offsets, pairs, k, limit=0.0):
    """(y fp32 [P, H] before its rounding, by pair; gate, up, h float64 [P, I] by sorted row)."""
    P, I = len(pairs), w13.shape[1] // 2
    y = np.zeros((P, w2.shape[1]), np.float32)
    gate, up, hid = (np.zeros((P, I)) for _ in range(3))
    for e in range(w13.shape[0]):
        rows = np.arange(offsets[e], offsets[e + 1])
        if not len(rows):
            continue
        gu = linear32(x_bits[pairs[rows] // k], w13[e], s13[e]).astype(np.float64)
        g, u = gu[:, :I], gu[:, I:]
        if limit > 0:
            g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
        gate[rows], up[rows] = g, u
        with np.errstate(over="ignore"):
            hid[rows] = g / (1.0 + np.exp(-g)) * u
        y[pairs[rows]] = linear32(codecs.bf16_encode(hid[rows].astype(np.float32)), w2[e], s2[e])
    return y, gate, up, hid
