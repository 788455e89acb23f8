"""Router losses and gradient: workspaces that serve several batches, rows outside of every sequence, many sequences.

Tolerances: those of test_gpu_router_training, where they are derived."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
import test_gpu_router_training as tr
from oracle import router

pytestmark = pytest.mark.gpu


def test_workspace_of_the_largest_batch():
    """The bytes for 16385 tokens, whose chunks are longer, serve 16384 tokens (more chunks) and fewer."""
    d, (E, k, S), most = gh.dev(), (8, 2, 3), 16385
    ws = torch.empty(lib.moe_balance_loss_workspace_bytes(most, E, S), dtype=torch.uint8, device=d)
    for T in (16385, 16384, 129, 5):
        _, logits, ids, off, _ = tr._case(T, E, k, S, False, 21)
        loss, counts = torch.full((2,), 9.0, device=d), torch.full((S, E), -1, dtype=torch.int32, device=d)
        tokens = torch.full((S,), -1, dtype=torch.int32, device=d)
        ws.fill_(0xFF)
        lib.moe_balance_loss(T, E, k, tr._dev(logits), tr._dev(ids), loss, counts, tokens, ws, 0.01, 0.001, num_seqs=S,
                             seq_offsets=tr._dev(off))
        torch.cuda.synchronize()
        rl, rc, rt = router.balance_loss(logits, ids, 0.01, 0.001, None, off)
        assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
        assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= tr.TOL * np.abs(rl))


@pytest.mark.parametrize("T", [50, 700])
def test_rows_in_no_sequence_have_no_part(T):
    """Rows before the first sequence and behind the last one, which hold anything: nothing reaches the losses, and
    their gradient is that through the weights alone."""
    rng, logits, ids, _, _ = tr._case(T, 200, 4, 1, False, 22)
    off = np.array([9, 9, 30, T - 11], np.int32)
    out = np.r_[0:9, T - 11:T]
    w, dw = rng.random(ids.shape).astype(np.float32), rng.standard_normal(ids.shape).astype(np.float32)
    dl = np.array([1.0, -0.5], np.float32)
    a = tr._loss(logits, ids, off, None, 0.5, 0.25)
    ga = tr._grad(logits, ids, off, None, 0.5, 0.25, w, dw, dl, a[1], a[2])
    la = tr._grad(logits, ids, off, None, 0.5, 0.25, None, None, dl, a[1], a[2])
    assert not la[out].any()
    for bad in (np.nan, np.inf, -np.inf, np.finfo(np.float32).max):
        logits[out] = bad
        b = tr._loss(logits, ids, off, None, 0.5, 0.25)
        assert all(torch.equal(x, y) for x, y in zip(a, b)), bad
        assert np.array_equal(ga, tr._grad(logits, ids, off, None, 0.5, 0.25, w, dw, dl, a[1], a[2])), bad
        assert np.array_equal(la, tr._grad(logits, ids, off, None, 0.5, 0.25, None, None, dl, a[1], a[2])), bad


@pytest.mark.parametrize("T,E,k,S", [(3000, 64, 6, 1000), (90, 256, 8, 5000), (300, 33, 2, 65536)])
def test_many_sequences(T, E, k, S):
    """Hundreds of sequences and more, most of them of a few tokens or none."""
    rng, logits, ids, off, mask = tr._case(T, E, k, S, True, 23)
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    loss, counts, tokens = tr._loss(logits, ids, off, mask, 0.01, 0.001)
    rl, rc, rt = router.balance_loss(logits, ids, 0.01, 0.001, mask, off)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= tr.TOL * np.abs(rl))
    again = tr._loss(logits, ids, off, mask, 0.01, 0.001)
    assert torch.equal(again[0], loss)
    w, dw = rng.random(ids.shape).astype(np.float32), rng.standard_normal(ids.shape).astype(np.float32)
    ref, mag = router.backward(logits, ids, w, dw, (1.0, 1.0), 0.01, 0.001, mask, off)
    g = tr._grad(logits, ids, off, mask, 0.01, 0.001, w, dw, np.ones(2, np.float32), counts, tokens)
    assert np.all(np.abs(g - ref) <= tr.TOL * mag)


def test_offsets_beyond_32_bits():
    """Logits of over 2^31 values: the losses and counts of all of them, the gradient's first and last rows, and those
    around 2^31 values, against torch in float64."""
    d, (T, E, k) = gh.dev(), ((1 << 21) + 5, 1024, 2)
    g = torch.Generator(device=d)
    g.manual_seed(24)
    logits = torch.empty(T, E, device=d)
    logits.normal_(generator=g)
    ids = torch.randint(0, E, (T, k), generator=g, device=d, dtype=torch.int32)
    loss, counts = torch.empty(2, device=d), torch.empty(1, E, dtype=torch.int32, device=d)
    tokens = torch.empty(1, dtype=torch.int32, device=d)
    ws = torch.empty(lib.moe_balance_loss_workspace_bytes(T, E), dtype=torch.uint8, device=d)
    lib.moe_balance_loss(T, E, k, logits, ids, loss, counts, tokens, ws, 0.01, 0.001)
    P, z = torch.zeros(E, dtype=torch.float64, device=d), 0.0
    for t in range(0, T, 1 << 17):
        v = logits[t:t + (1 << 17)].double()
        P += torch.softmax(v, 1).sum(0)
        z += float(torch.logsumexp(v, 1).square().sum())
    c = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(counts[0].long(), c) and int(tokens) == T
    ref = [0.01 * float((E * c.double() / (k * T) * P / T).sum()), 0.001 * z / T]
    assert all(abs(a - b) <= tr.TOL * abs(b) for a, b in zip(loss.tolist(), ref))
    out = torch.empty(T, E, device=d)
    lib.moe_route_backward(T, E, k, logits, ids, out, d_loss=torch.ones(2, device=d), counts=counts, tokens=tokens,
                           balance_coef=0.01, z_coef=0.001)
    torch.cuda.synchronize()
    f = 0.01 / T * (E * c.double() / (k * T) - 1.0)
    for t in (0, (1 << 21) - 4, T - 8):
        v = logits[t:t + 8].double()
        p, zt = torch.softmax(v, 1), 2e-3 / T * torch.logsumexp(v, 1)[:, None]
        want = p * (f - (p * f).sum(1, keepdim=True)) + zt * p
        mag = p * (f.abs() + (p * f.abs()).sum(1, keepdim=True) + zt.abs())
        assert bool(((out[t:t + 8].double() - want).abs() <= tr.TOL * mag).all()), t
