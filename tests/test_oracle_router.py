"""Pins of the router's loss and gradient oracle: torch autograd in float64,
central differences, and closed forms."""
import numpy as np
import pytest
import torch

from oracle import router


def _case(T=13, E=7, k=3, S=3, seed=0):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E)) * 2
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    off = np.array([0, 4, 4, T])[: S + 1] if S == 3 else np.array([0, T])
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    return rng, logits, ids, off, mask


def _torch_loss(z, ids, mask, off, coef, zc):
    E, k, S = z.shape[1], ids.shape[1], len(off) - 1
    out = z.new_zeros(2)
    for s in range(S):
        rows = [t for t in range(off[s], off[s + 1]) if mask[t]]
        if not rows:
            continue
        p, n = torch.softmax(z[rows], 1), len(rows)
        c = torch.bincount(torch.from_numpy(ids[rows].reshape(-1)).long(), minlength=E).double()
        out = out + torch.stack([coef / S * (E * c / (k * n) * p.mean(0)).sum(),
                                 zc / S * torch.logsumexp(z[rows], 1).square().mean()])
    return out


def test_loss_and_gradient_are_autograds():
    rng, logits, ids, off, mask = _case()
    z = torch.from_numpy(logits).requires_grad_()
    loss = _torch_loss(z, ids, mask, off, 0.3, 0.2)
    got, counts, tokens = router.balance_loss(logits, ids, 0.3, 0.2, mask, off)
    assert np.allclose(got, loss.detach().numpy(), rtol=1e-12)
    assert tokens.sum() == mask.sum() and counts.sum() == 3 * mask.sum() and tokens[1] == 0
    dw = rng.standard_normal(ids.shape) * mask[:, None]
    w = torch.softmax(torch.gather(z, 1, torch.from_numpy(ids).long()), 1)
    (1.5 * loss[0] - 0.5 * loss[1] + (w * torch.from_numpy(dw)).sum()).backward()
    d, mag = router.backward(logits, ids, w.detach().numpy(), dw, (1.5, -0.5), 0.3, 0.2, mask, off)
    assert np.allclose(d, z.grad.numpy(), rtol=1e-10, atol=1e-14)
    assert np.all(np.abs(d) <= mag * (1 + 1e-12))


def test_gradient_is_the_differences():
    _, logits, ids, off, mask = _case(T=9, E=5, k=2, seed=1)
    off = np.array([0, 4, 4, 9])
    d, _ = router.backward(logits, ids, None, None, (1.0, 1.0), 0.5, 0.1, mask, off)
    h = 1e-5
    for t in range(9):
        for e in range(5):
            up, dn = logits.copy(), logits.copy()
            up[t, e] += h
            dn[t, e] -= h
            diff = (router.balance_loss(up, ids, 0.5, 0.1, mask, off)[0].sum()
                    - router.balance_loss(dn, ids, 0.5, 0.1, mask, off)[0].sum()) / (2 * h)
            assert abs(diff - d[t, e]) < 1e-9


def test_even_routing_has_the_least_loss():
    """f = 1 for every expert: the loss is coef whatever the logits, its gradient zero."""
    E, k = 6, 2
    ids = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    logits = np.random.default_rng(2).standard_normal((3, E))
    loss, _, _ = router.balance_loss(logits, ids, 0.7, 0.0)
    assert loss[0] == pytest.approx(0.7, rel=1e-14)
    d, _ = router.backward(logits, ids, None, None, (1.0, 0.0), 0.7, 0.0)
    assert np.abs(d).max() < 1e-15


def test_ids_outside_are_not_counted_and_twice_is_twice():
    ids = np.array([[-1, 2], [2, 2], [9, 0]], np.int32)
    _, counts, tokens = router.balance_loss(np.zeros((3, 4)), ids, 1.0, 0.0)
    assert counts.tolist() == [[1, 0, 3, 0]] and tokens.tolist() == [3]
    d, _ = router.backward(np.zeros((3, 4)), ids, np.full((3, 2), 0.5), np.ones((3, 2)) * [[1.0, 3.0]])
    assert np.allclose(d[0], [0, 0, 0.5 * (3 - 2), 0]) and np.allclose(d[1], [0, 0, 0.5 * (1 - 2 + 3 - 2), 0])
