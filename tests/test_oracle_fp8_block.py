"""Pins of the block-128 fp8 oracle: codes against torch's e4m3 cast and a
brute-force nearest search, scales by hand, products against dense ones."""
import numpy as np
import pytest
import torch

from oracle import codecs, fp8_block as fb, moe


def test_codes_are_torchs_cast():
    rng = np.random.default_rng(0)
    x = codecs.bf16_decode(codecs.bf16_encode((rng.standard_normal((9, 300)) * 3).astype(np.float32))).astype(np.float32)
    c, s = fb.quantize_rows(x)
    b = torch.nn.functional.pad(torch.from_numpy(x), (0, 384 - 300)).view(9, 3, 128)
    amax = b.abs().amax(2, keepdim=True)
    want = (b * (torch.full_like(amax, 448.0) / amax)).to(torch.float8_e4m3fn).view(torch.uint8).view(9, 384)[:, :300]
    assert np.array_equal(c, want.numpy())
    assert np.array_equal(s, (amax / torch.full_like(amax, 448.0))[..., 0].numpy())


def test_largest_value_gets_the_largest_code_and_zero_rows_stay_zero():
    x = np.zeros((2, 256), np.float32)
    x[0, 5], x[0, 200] = -3.0, 1e-3
    c, s = fb.quantize_rows(x)
    assert c[0, 5] == 0xFE and c[0, 200] == 0x7E and not c[1].any()
    assert s[0, 0] == np.float32(3.0 / 448) and s[1, 0] == np.float32(2.0 ** -100) / np.float32(448)
    assert np.allclose(fb.dequantize_rows(c, s), x, rtol=2.0 ** -23)


def test_weight_blocks_are_ragged():
    rng = np.random.default_rng(1)
    w = (rng.standard_normal((130, 144)) * 0.02).astype(np.float32)
    c, s = fb.quantize_weights(w)
    assert s.shape == (2, 2)
    assert s[1, 1] == np.abs(w[128:, 128:]).max() / np.float32(448)
    # half a step of e4m3 (2^-4 of a normal value), or half the subnormal quantum of the block's scale
    err = np.abs(fb.dequantize_weights(c, s) - w)
    step = np.repeat(np.repeat(s, 128, 0)[:130], 128, 1)[:, :144]
    assert np.all(err <= np.maximum(np.abs(w) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -20))


def test_representable_product_is_exact():
    """Values that are code * power of two, a largest magnitude of 448 in each block: nothing is rounded."""
    rng = np.random.default_rng(2)
    vals = codecs.e4m3_decode(np.arange(0x40, 0x7F, dtype=np.uint8))
    x = rng.choice(vals, (3, 256)).astype(np.float32)
    x[:, ::128] = 448.0
    w = rng.choice(vals, (5, 256)).astype(np.float32)
    w[0, ::128] = 448.0
    y, _ = fb.linear(codecs.bf16_encode(x), *fb.quantize_weights(w))
    assert np.array_equal(y, x.astype(np.float64) @ w.astype(np.float64).T)


@pytest.mark.parametrize("limit", [0.0, 0.5])
def test_experts_are_the_dense_mlp_of_each_pair(limit):
    rng = np.random.default_rng(3)
    T, H, I, E, k = 6, 256, 128, 4, 2
    x = codecs.bf16_encode(rng.standard_normal((T, H)).astype(np.float32))
    q13 = [fb.quantize_weights((rng.standard_normal((2 * I, H)) * 0.1).astype(np.float32)) for _ in range(E)]
    q2 = [fb.quantize_weights((rng.standard_normal((H, I)) * 0.1).astype(np.float32)) for _ in range(E)]
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    y = fb.experts(x, ids, np.stack([c for c, _ in q13]), np.stack([s for _, s in q13]),
                   np.stack([c for c, _ in q2]), np.stack([s for _, s in q2]), limit)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            gu = fb.linear(x[t:t + 1], *q13[e])[0]
            h = codecs.bf16_encode(moe.silu_mul(gu[:, :I], gu[:, I:], limit).astype(np.float32))
            assert np.allclose(y[t * k + j], fb.linear(h, *q2[e])[0][0], rtol=1e-12)
