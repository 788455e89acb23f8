"""Experts on block-128 fp8 weights at the ends of their range, row by row, and the few-token path's exact sums.

Tolerances: over all values those of test_gpu_fp8 (6e-3).  A row or a 128-column block by itself: where the gate and up
sums' error carries a block's largest intermediate value over a bf16 border, the block's scale moves and all of its
values are quantised anew, each within half a step (2^-4) of e4m3 both times: evenly spread, sqrt(2) 2^-4 / sqrt(3) =
5.1e-2 of them in the root mean square, and the output's rounding (2.3e-3) beside it, below 2^-4.  A row or block that
is wrong is off by its own size."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
import test_gpu_fp8 as t8
from oracle import codecs, fp8_block as fb

pytestmark = pytest.mark.gpu


def _run(x, ids, w, E, limit=0.0):
    """y float64 [T k, H] through moe_permute and moe_fp8_experts; w numpy arrays."""
    d, (T, H), k, I = gh.dev(), x.shape, ids.shape[1], w[0].shape[1] // 2
    shape = lib.make_shape(H, I, E, k, T, "bf16", gate_up_limit=limit)
    off = torch.empty(E + 1, dtype=torch.int32, device=d)
    pairs, pos = (torch.empty(T * k, dtype=torch.int32, device=d) for _ in range(2))
    xd = gh.to_device_x(x)
    lib.moe_permute(shape, T, torch.from_numpy(ids).to(d), xd, off, pairs, pos, xd)
    y = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device=d)
    ws = torch.full((lib.moe_fp8_experts_workspace_bytes(shape),), 0xFF, dtype=torch.uint8, device=d)
    lib.moe_fp8_experts(shape, T, *(torch.from_numpy(v).to(d) for v in w), off, pairs, xd, y, ws)
    torch.cuda.synchronize()
    return y.double().cpu().numpy()


@pytest.mark.parametrize("T,H,I,E,k,limit", [(1, 640, 256, 8, 8, 0.0), (8, 1152, 384, 30, 6, 0.1), (7, 8192, 128, 4, 2, 0.0),
                                             (50, 640, 256, 4, 2, 0.0), (333, 384, 128, 9, 3, 0.1),
                                             (700, 896, 256, 3, 2, 0.0)])
def test_experts_row_by_row(T, H, I, E, k, limit):
    rng = np.random.default_rng(T + 5 * H)
    x, w = t8._x(rng, T, H), t8._layer(rng, H, I, E)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    got, ref = _run(x, ids, w, E, limit), fb.experts(x, ids, *w, limit)
    err = got - ref
    assert np.linalg.norm(err) <= 6e-3 * np.linalg.norm(ref)
    rows = np.linalg.norm(err, axis=1) / np.linalg.norm(ref, axis=1)
    blocks = np.linalg.norm(err.reshape(T * k, -1, 128), axis=2) / np.linalg.norm(ref.reshape(T * k, -1, 128), axis=2)
    print(f"  T={T} H={H}: worst row {rows.max():.2e}, worst block {blocks.max():.2e}", flush=True)
    assert rows.max() <= 2.0 ** -4 and blocks.max() <= 2.0 ** -4


@pytest.mark.parametrize("T,H", [(1, 256), (3, 1024), (8, 512), (8, 8192)])
def test_gate_up_sums_of_few_tokens_are_exact(T, H):
    """Products of 2^16 that cancel inside a group of eight, beside products of 14: a sum that cuts products at the
    group's largest would count those as 8, and be off by almost half."""
    rng, I, E, k = np.random.default_rng(T + H), 128, 6, 3
    big, small = codecs.e4m3_encode(np.float32([256.0]))[0], codecs.e4m3_encode(np.float32([3.75]))[0]
    c13 = np.zeros((E, 2 * I, H), np.uint8)
    s13 = np.full((E, 2 * I // 128, H // 128), np.float32(2.0 ** -4))
    c13[:, :, 0::8], c13[:, :, 1::8], c13[:, :, 2::8] = big, big | 0x80, small
    c13[:, I:, 2::8] ^= (rng.random((E, I, H // 8)) < 0.5).astype(np.uint8) << 7
    _, _, w2, s2 = t8._layer(rng, 128, I, E)
    w2, s2 = np.tile(w2, (1, H // 128, 1)), np.tile(s2, (1, H // 128, 1))
    x = np.zeros((T, H), np.float32)  # largest magnitude 448 in each block: scale 1, codes as they stand
    x[:, 0::8], x[:, 1::8], x[:, 2::8] = 256.0, 256.0, 3.75
    x[:, 7::128] = 448.0
    x[:, 2::8] *= np.where(rng.random((T, H // 8)) < 0.9, 1.0, -1.0)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    bits = codecs.bf16_encode(x)
    got, ref = _run(bits, ids, (c13, s13, w2, s2), E), fb.experts(bits, ids, c13, s13, w2, s2)
    rows = np.linalg.norm(got - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert rows.max() <= 6e-3, rows


@pytest.mark.parametrize("T", [2047, 2048])
def test_experts_offsets_beyond_32_bits(T):
    """x of 2^31 values and just below: the streaming kernel and the tiled one, whose gathered rows have 32-bit addresses.
    The first and last rows against a float64 product on the same codes."""
    d, (H, I) = gh.dev(), (1 << 20, 128)
    g = torch.Generator(device=d)
    g.manual_seed(T)
    w13, w2 = (torch.randint(0, 256, s, generator=g, device=d, dtype=torch.uint8) for s in ((2 * I, H), (H, I)))
    for w in (w13, w2):
        w[(w & 0x7F) == 0x7F] = 0x30
    s13 = 1e-5 * (0.5 + torch.rand(2, H // 128, generator=g, device=d))
    s2 = 1e-4 * (0.5 + torch.rand(H // 128, 1, generator=g, device=d))
    x = torch.empty(T, H, dtype=torch.bfloat16, device=d)
    for t in range(0, T, 256):
        x[t:t + 256] = torch.randn(x[t:t + 256].shape, generator=g, device=d)
    shape = lib.make_shape(H, I, 1, 1, T, "bf16")
    off = torch.tensor([0, T], dtype=torch.int32, device=d)
    pairs = torch.arange(T, dtype=torch.int32, device=d)
    y = torch.empty(T, H, dtype=torch.bfloat16, device=d)
    ws = torch.empty(lib.moe_fp8_experts_workspace_bytes(shape), dtype=torch.uint8, device=d)
    lib.moe_fp8_experts(shape, T, w13, s13, w2, s2, off, pairs, x, y, ws)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=d)

    def rows64(bits):
        return torch.from_numpy(fb.dequantize_rows(*fb.quantize_rows(codecs.bf16_decode(bits)))).to(d)

    def product(v, w, s):
        o = torch.empty(v.shape[0], w.shape[0], dtype=torch.float64, device=d)
        for n in range(0, w.shape[0], 128):  # one row of scales
            o[:, n:n + 128] = v @ (w[n:n + 128].view(torch.float8_e4m3fn).double()
                                   * s[n // 128].double().repeat_interleave(128)).t()
        return o

    gu = product(rows64(gh.bf16_numpy(x[pick])), w13, s13)
    h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    ref = product(rows64(gh.bf16_numpy(h.float().to(torch.bfloat16))), w2, s2)
    err = (y[pick].double() - ref).norm(dim=1) / ref.norm(dim=1)
    print(f"  T={T}: rows off by {err.tolist()}", flush=True)
    assert bool((err <= 2.0 ** -4).all())
