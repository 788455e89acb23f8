"""Expert MLPs on 8-bit weights whose intermediate is certain, so that every output is
compared bit for bit.

The gates are all above 40: exp(-g) is lost in 1 + exp(-g) in 32 bits and in 64, silu(g)
is g, and h is bf16(fp32(g u)), one product of two fp32 numbers, the same in both.  All
else is integers and the definition's roundings.  (With ordinary gates an h may lie on a
border between two bf16 values, and over a long down product every row has one that does.)"""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import codecs, int8

pytestmark = pytest.mark.gpu


def _case(T, H, I, E, k, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H)).astype(np.float32)
    x[:, 0] = 16.0  # the row's largest value: code 127
    w13 = rng.integers(-127, 128, (E, 2 * I, H)).astype(np.int8)
    w13[:, :I] = rng.integers(-2, 3, (E, I, H))
    w13[:, :I, 0] = 127
    # a gate's sum is 127 127 and a rest of less than a third of it: g about 60
    s13 = (rng.random((E, 2 * I)) * 1e-3 + 1e-4).astype(np.float32)
    s13[:, :I] = 60 / (127 * 127 * 16 / 127)
    w2 = rng.integers(-127, 128, (E, H, I)).astype(np.int8)
    s2 = (rng.random((E, H)) * 1e-3 + 1e-4).astype(np.float32)
    ids = np.argsort(-(rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)), axis=1, kind="stable")[:, :k].reshape(-1)
    off = np.r_[0, np.cumsum(np.bincount(ids, minlength=E))].astype(np.int32)
    return codecs.bf16_encode(x), w13, s13, w2, s2, off, np.argsort(ids, kind="stable").astype(np.int32)


def _run(c, k, limit):
    x, w13, s13, w2, s2, off, pairs = c
    d, (T, H), (E, I) = gh.dev(), x.shape, (w13.shape[0], w2.shape[2])
    shape = lib.make_shape(H, I, E, k, T, "bf16", gate_up_limit=limit)
    ws = torch.full((lib.moe_int8_experts_workspace_bytes(shape),), 0xFF, dtype=torch.uint8, device=d)
    y = torch.full((T * k + 1, H), 7.0, dtype=torch.bfloat16, device=d)
    lib.moe_int8_experts(shape, T, *(torch.from_numpy(v).to(d) for v in c[1:]), gh.to_device_x(x), y, ws)
    torch.cuda.synchronize()
    assert (y[T * k] == 7.0).all()
    return y[:T * k].view(torch.int16).cpu().numpy().view(np.uint16)


# K of the down product past 8192 values (a row is read twice by its quantiser) and of few steps; one token to the largest
# tiles; rows of a wave and of a block
@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 256, 16640, 4, 2), (6, 256, 16640, 4, 2), (60, 256, 16640, 4, 2), (150, 128, 16640, 4, 2), (400, 128, 16640, 4, 2),
    (12, 128, 8320, 16, 3), (600, 128, 8320, 5, 2), (3, 512, 768, 60, 4), (64, 512, 768, 60, 4), (333, 512, 384, 16, 3),
    (700, 384, 512, 6, 2), (1100, 256, 1408, 8, 2), (16, 4096, 256, 8, 2)])
def test_every_output_bit(T, H, I, E, k):
    c = _case(T, H, I, E, k, T + I)
    x, w13, s13, w2, s2, off, pairs = c
    for limit in (0.0, 50.0):  # (a clamp that every gate reaches and few up values)
        y, gate, up, hid = int8.experts(x, w13, s13, w2, s2, off, pairs, k, limit)
        assert gate.min() > 40 and np.isfinite(hid).all()
        ref = codecs.bf16_encode(y)
        assert (ref & 0x7FFF != 0).mean() > 0.99
        got = _run(c, k, limit)
        assert np.array_equal(got, ref), (limit, np.argwhere(got != ref)[:4], (got != ref).mean())
