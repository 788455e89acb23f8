"""Balance loss, router z-loss and the gradient of the router's logits
(oracle; test infrastructure): per-token loops over the definitions, float64.
"""
from __future__ import annotations

import numpy as np


def _softmax(row):
    m = row.max()
    e = np.exp(row - m)
    return e / e.sum(), m + np.log(e.sum())


def balance_loss(logits, ids, coef, z_coef, mask=None, seq_offsets=None):
    """(loss float64 [2], counts int [S, E], tokens int [S])."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k = ids.shape[1]
    off = [0, T] if seq_offsets is None else list(seq_offsets)
    S = len(off) - 1
    loss, counts, tokens = np.zeros(2), np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    for s in range(S):
        P, z = np.zeros(E), 0.0
        for t in range(off[s], off[s + 1]):
            if mask is not None and not mask[t]:
                continue
            p, lse = _softmax(logits[t])
            P += p
            z += lse * lse
            tokens[s] += 1
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        n = tokens[s]
        if n:
            loss[0] += coef / S * float(((E * counts[s] / (k * n)) * (P / n)).sum())
            loss[1] += z_coef / S * z / n
    return loss, counts, tokens


def backward(logits, ids, topk_w=None, d_topk_w=None, d_loss=None, coef=0.0, z_coef=0.0, mask=None,
             seq_offsets=None):
    """(d_logits float64 [T, E], magnitude [T, E]: the sum of the magnitudes of the terms of each value)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k = ids.shape[1]
    off = [0, T] if seq_offsets is None else list(seq_offsets)
    S = len(off) - 1
    _, counts, tokens = balance_loss(logits, ids, 0.0, 0.0, mask, seq_offsets) if d_loss is not None else (0, 0, 0)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        if d_loss is not None:
            s = next((i for i in range(S) if off[i] <= t < off[i + 1]), None)
            if s is not None:
                p, lse = _softmax(logits[t])
                n = tokens[s]
                f = d_loss[0] * coef / (S * n) * (E * counts[s] / (k * n) - 1.0)
                z = d_loss[1] * z_coef * 2.0 / (S * n) * lse
                d[t] += p * (f - (p * f).sum()) + z * p
                mag[t] += p * (np.abs(f) + (p * np.abs(f)).sum() + abs(z))
        if d_topk_w is not None:
            w, dw = np.asarray(topk_w[t], np.float64), np.asarray(d_topk_w[t], np.float64)
            dot, adot = (w * dw).sum(), np.abs(w * dw).sum()
            for j, e in enumerate(ids[t]):
                if 0 <= e < E:
                    d[t, e] += w[j] * (dw[j] - dot)
                    mag[t, e] += abs(w[j]) * (abs(dw[j]) + adot)
    return d, mag
