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
