"""Routing by scores and its gradient (oracle; test infrastructure): token by
token, float64, with the fp32 roundings that the definition names.
"""
from __future__ import annotations

import numpy as np

NEG = np.float32(-np.inf)


def scores(row, kind):
    """Scores of one token's logits, float64; experts at -inf have 0."""
    row = np.asarray(row, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return np.array([1.0 / (1.0 + np.exp(-v)) if v >= 0 else np.exp(v) / (1.0 + np.exp(v)) for v in row])
        m = row.max()
        if m == -np.inf:
            return np.zeros_like(row)
        e = np.exp(row - m)
        return e / e.sum()


def shares(z, kind):
    """Scores of the picks with logits z over their sum, by the scores' logarithms: where the scores themselves leave the
    64-bit numbers too; 0 where every pick is off."""
    z = np.asarray(z, np.float64)
    if not len(z) or z.max() == -np.inf:
        return np.zeros_like(z)
    v = -np.logaddexp(0.0, -z) if kind == "sigmoid" else z  # a softmax's sum is the same for all picks
    e = np.exp(v - v.max())
    return e / e.sum()


def _ranked(values):
    """Positions by value, largest first, equal ones in order."""
    return sorted(range(len(values)), key=lambda i: (-float(values[i]), i))


def route(logits, k, kind, bias=None, groups=1, kept=1, top=1, renorm=True, scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k])."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    per = E // groups
    ids, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        s = scores(logits[t], kind)
        c = s.astype(np.float32)
        if bias is not None:
            c = c + np.asarray(bias, np.float32)
        c = np.where(logits[t] == NEG, NEG, c).astype(np.float32)
        best = [np.sort(c[g * per:(g + 1) * per])[::-1][:top] for g in range(groups)]
        total = [b[0] if top == 1 else np.float32(b[0] + b[1]) for b in best]
        mine = sorted(_ranked(total)[:kept])
        cand = [e for g in mine for e in range(g * per, (g + 1) * per)]
        ids[t] = [cand[i] for i in _ranked(c[cand])[:k]]
        w[t] = scale * (shares(logits[t, ids[t]], kind) if renorm else s[ids[t]])
    return ids, w


def backward(logits, ids, d_w, kind, renorm=True, scale=1.0, mask=None):
    """(d_logits float64 [T, E], magnitude: the sum of the magnitudes of the terms of each value)."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        s = scores(logits[t], kind)
        ok = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        g = scale * np.asarray(d_w[t], np.float64)
        v = shares([logits[t, ids[t, j]] for j in ok], kind) if renorm else s[ids[t, ok]]  # in the order of ok
        dot = adot = 0.0
        if renorm:
            dot = sum(g[j] * v[i] for i, j in enumerate(ok))
            adot = sum(abs(g[j]) * v[i] for i, j in enumerate(ok))
        for i, j in enumerate(ok):
            e = ids[t, j]
            z = float(logits[t, e])
            # of the weight by its own logit, but for the sum's part
            dv = v[i] if kind == "softmax" else v[i] * (1.0 / (1.0 + np.exp(z)) if z < 0 else np.exp(-z) / (1.0 + np.exp(-z)))
            d[t, e] += (g[j] - dot) * dv
            mag[t, e] += (abs(g[j]) + adot) * dv
        if kind == "softmax" and not renorm:
            dot = sum(g[j] * s[ids[t, j]] for j in ok)
            d[t] -= s * dot
            mag[t] += s * sum(abs(g[j]) * s[ids[t, j]] for j in ok)
    return d, mag
