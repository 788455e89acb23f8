"""Block-128 fp8 products whose operands end where their memory ends: tiles that are not full read nothing behind it.

Tolerances: those of the same products elsewhere (test_gpu_fp8)."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
import test_gpu_fp8 as t8
from oracle import fp8_block as fb

pytestmark = pytest.mark.gpu


def _at_the_end(nbytes):
    """nbytes u8 that end with an allocation of its own (large ones are whole 2 MiB pages)."""
    whole = -(-(nbytes + (64 << 20)) >> 21) << 21
    return torch.full((whole,), 0xFF, dtype=torch.uint8, device=gh.dev())[whole - nbytes:]


def _put(v):
    v = np.ascontiguousarray(v)
    o = _at_the_end(v.nbytes)
    o.copy_(torch.from_numpy(v.reshape(-1).view(np.uint8)).to(o.device))
    return o


# partly filled tiles of every shape: few and many of them, one row or one weight row in the last one
@pytest.mark.parametrize("M,N,K", [(33, 129, 272), (65, 257, 1040), (200, 1025, 400), (129, 2817, 4096), (500, 2000, 144),
                                   (1000, 2901, 144), (2049, 4097, 272), (1793, 3850, 1024)])
def test_linear_at_the_end_of_memory(M, N, K):
    rng = np.random.default_rng(M + N + K)
    x, (c, s) = t8._x(rng, M, K), t8._weights(rng, N, K)
    out = _at_the_end(2 * M * N)
    ws = _at_the_end(lib.moe_fp8_linear_workspace_bytes(M, N, K))
    lib.moe_fp8_linear(M, N, K, _put(c), _put(s), _put(x), out, ws)
    torch.cuda.synchronize()
    got = out.view(torch.bfloat16).view(M, N).double().cpu().numpy()
    t8._check(got, *fb.linear(x, c, s))


@pytest.mark.parametrize("T,H,I,E,k", [(40, 384, 256, 2, 1), (70, 128, 384, 3, 2), (300, 384, 256, 5, 2),
                                       (700, 640, 128, 3, 2)])
def test_experts_at_the_end_of_memory(T, H, I, E, k):
    """An H that is not a multiple of the tiles' 256 weight rows: the last expert's last tile is half empty."""
    rng, d = np.random.default_rng(T + H), gh.dev()
    x, w = t8._x(rng, T, H), t8._layer(rng, H, I, E)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    shape = lib.make_shape(H, I, E, k, T, "bf16")
    off = torch.empty(E + 1, dtype=torch.int32, device=d)
    pairs, pos = (torch.empty(T * k, dtype=torch.int32, device=d) for _ in range(2))
    xd = _put(x)
    lib.moe_permute(shape, T, torch.from_numpy(ids).to(d), xd, off, pairs, pos, xd)
    y = _at_the_end(2 * T * k * H)
    ws = _at_the_end(lib.moe_fp8_experts_workspace_bytes(shape))
    lib.moe_fp8_experts(shape, T, *(_put(v) for v in w), off, pairs, xd, y, ws)
    torch.cuda.synchronize()
    ref = fb.experts(x, ids, *w)
    got = y.view(torch.bfloat16).view(T * k, H).double().cpu().numpy()
    assert np.linalg.norm(got - ref) <= 6e-3 * np.linalg.norm(ref)
