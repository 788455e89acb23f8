"""Products on block-128 fp8 weights (oracle; test infrastructure).

Weights: e4m3fn codes [N, K] with one fp32 scale per 128 x 128 block.
Activations: bf16 rows, one fp32 scale per row and 128 columns:
amax = max(max |x|, 2^-100), scale = fp32(amax / 448), code =
e4m3(fp32(x * fp32(448 / amax))).  Products and sums in float64.
"""
from __future__ import annotations

import numpy as np

from . import codecs, moe

BLK = 128
TINY = np.float32(2.0 ** -100)


def _blocks(n):
    return -(-n // BLK)


def quantize_rows(x32):
    """(codes u8 [R, K], scales fp32 [R, ceil(K / 128)]) of finite fp32 rows."""
    x32 = np.asarray(x32, np.float32)
    R, K = x32.shape
    codes = np.zeros((R, K), np.uint8)
    scales = np.zeros((R, _blocks(K)), np.float32)
    for b in range(_blocks(K)):
        v = x32[:, b * BLK:(b + 1) * BLK]
        amax = np.maximum(np.abs(v).max(axis=1), TINY).astype(np.float32)
        scales[:, b] = amax / np.float32(448)
        codes[:, b * BLK:(b + 1) * BLK] = codecs.e4m3_encode(v * (np.float32(448) / amax)[:, None])
    return codes, scales


def quantize_weights(w32):
    """(codes u8 [N, K], scales fp32 [ceil(N / 128), ceil(K / 128)]) of an fp32 matrix."""
    w32 = np.asarray(w32, np.float32)
    N, K = w32.shape
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((_blocks(N), _blocks(K)), np.float32)
    for i in range(_blocks(N)):
        for j in range(_blocks(K)):
            at = np.s_[i * BLK:(i + 1) * BLK, j * BLK:(j + 1) * BLK]
            amax = np.float32(max(np.abs(w32[at]).max(), TINY))
            scales[i, j] = amax / np.float32(448)
            codes[at] = codecs.e4m3_encode(w32[at] * (np.float32(448) / amax))
    return codes, scales


def dequantize_rows(codes, scales):
    K = codes.shape[1]
    return codecs.e4m3_decode(codes).astype(np.float64) * np.repeat(scales.astype(np.float64), BLK, 1)[:, :K]


def dequantize_weights(codes, scales):
    N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), BLK, 0)[:N], BLK, 1)[:, :K]
    return codecs.e4m3_decode(codes).astype(np.float64) * s


def _group_max(v):
    """Largest magnitude of every 8 consecutive columns, [R, ceil(K / 8)]."""
    R, K = v.shape
    full = np.zeros((R, -(-K // 8) * 8))
    full[:, :K] = np.abs(v)
    return full.reshape(R, -1, 8).max(axis=2)


def linear(x_bits, codes, scales):
    """float64 [M, N] before the output's rounding, and for each sum the sum over its groups of 8 consecutive products
    of a bound of the group's largest product (the product of the two operands' largest magnitudes)."""
    xh = dequantize_rows(*quantize_rows(codecs.bf16_decode(np.asarray(x_bits, np.uint16))))
    wh = dequantize_weights(codes, scales)
    return xh @ wh.T, _group_max(xh) @ _group_max(wh).T


def experts(x_bits, ids, w13, s13, w2, s2, limit=0.0):
    """y float64 [T k, H] (before the output's rounding) of each pair (t, j), p = t k + j."""
    T, k = ids.shape
    I = w13.shape[1] // 2
    y = np.zeros((T * k, w2.shape[1]))
    for e in np.unique(ids):
        p = np.flatnonzero(ids.reshape(-1) == e)
        gu, _ = linear(x_bits[p // k], w13[e], s13[e])
        h = codecs.bf16_encode(moe.silu_mul(gu[:, :I], gu[:, I:], limit).astype(np.float32))
        y[p], _ = linear(h, w2[e], s2[e])
    return y
