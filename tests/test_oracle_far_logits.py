"""Pins of the routing oracle's renormalised weights at logits whose scores leave the
64-bit numbers, by decimal arithmetic with wide exponents."""
import decimal

import numpy as np
import pytest

from oracle import scored_routing as sr


def _score(z, kind):
    with decimal.localcontext() as c:
        c.prec, c.Emin, c.Emax = 60, decimal.MIN_EMIN, decimal.MAX_EMAX
        e = decimal.Decimal(float(z)).exp()
        return e / (1 + e) if kind == "sigmoid" else e


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("base", [2.0, -5.0, -39.0, -41.0, -600.0, -703.0, -744.0, -760.0, -1.0e5, -2.0e8])
def test_shares(kind, base):
    rng = np.random.default_rng(3)
    z = (np.float32(base) + (2 * rng.standard_normal((6, 9))).astype(np.float32)).astype(np.float32)
    dw = rng.standard_normal((6, 4))
    bias = rng.standard_normal(9).astype(np.float32)
    ids, w = sr.route(z, 4, kind, bias, scale=2.5)
    d, mag = sr.backward(z, ids, dw, kind, True, 2.5)
    for t in range(6):
        s = [_score(z[t, e], kind) for e in ids[t]]
        with decimal.localcontext() as c:
            c.prec, c.Emin, c.Emax = 60, decimal.MIN_EMIN, decimal.MAX_EMAX
            v = [a / sum(s) for a in s]
            g = [decimal.Decimal(2.5) * decimal.Decimal(float(x)) for x in dw[t]]
            dot = sum(a * b for a, b in zip(g, v))
            for j, e in enumerate(ids[t]):
                assert abs(w[t, j] - 2.5 * float(v[j])) <= 1e-12 * w[t, j]
                rest = 1 - s[j] if kind == "sigmoid" else 1
                assert abs(d[t, e] - float((g[j] - dot) * v[j] * rest)) <= 1e-12 * mag[t, e]


def test_scores_go_down_to_the_smallest_numbers():
    s = sr.scores([-745.0, -720.0, -700.5, -100.0, 0.0, 800.0, -np.inf], "sigmoid")
    assert (s[:4] > 0).all() and s[4] == 0.5 and s[5] == 1.0 and s[6] == 0.0
    assert abs(s[2] / float(_score(-700.5, "sigmoid")) - 1) < 1e-12
