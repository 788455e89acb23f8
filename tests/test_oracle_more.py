"""Pins of the oracles of the scored routing, of the 8-bit integer products and of
an expert block's end: torch in float64 with autograd, closed forms and brute force."""
import numpy as np
import pytest
import torch

from oracle import block_end, codecs, int8, scored_routing as sr


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_is_torchs(kind, renorm):
    rng = np.random.default_rng(1)
    z = (rng.standard_normal((20, 24)) * 2).astype(np.float32)
    bias = (0.3 * rng.standard_normal(24)).astype(np.float32)
    ids, w = sr.route(z, 4, kind, bias, 6, 3, 2, renorm, 1.5)
    t = torch.from_numpy(z).double()
    s = torch.sigmoid(t) if kind == "sigmoid" else torch.softmax(t, 1)
    c = s.float() + torch.from_numpy(bias)
    g = c.view(20, 6, 4).topk(2, dim=2).values.sum(2).topk(3, dim=1).indices
    keep = torch.zeros(20, 6).scatter_(1, g, 1.0).repeat_interleave(4, 1).bool()
    ref = c.masked_fill(~keep, -np.inf).topk(4, dim=1).indices
    assert np.array_equal(ids, ref.numpy())
    v = s.gather(1, ref)
    v = 1.5 * (v / v.sum(1, keepdim=True) if renorm else v)
    assert np.allclose(w, v.numpy(), rtol=1e-13)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_gradient_is_autograds(kind, renorm):
    rng = np.random.default_rng(2)
    z = rng.standard_normal((9, 12)).astype(np.float32)
    ids = np.stack([rng.permutation(12)[:3] for _ in range(9)]).astype(np.int32)
    dw = rng.standard_normal((9, 3))
    mask = (np.arange(9) % 4 != 1).astype(np.uint8)
    t = torch.from_numpy(z).double().requires_grad_()
    s = torch.sigmoid(t) if kind == "sigmoid" else torch.softmax(t, 1)
    v = s.gather(1, torch.from_numpy(ids).long())
    v = 0.7 * (v / v.sum(1, keepdim=True) if renorm else v)
    (v * torch.from_numpy(dw * mask[:, None])).sum().backward()
    d, mag = sr.backward(z, ids, dw, kind, renorm, 0.7, mask)
    assert np.allclose(d, t.grad.numpy(), rtol=1e-12, atol=1e-15) and (mag >= np.abs(d) - 1e-15).all()


def test_routing_ties_and_switched_off_experts():
    z = np.zeros((3, 8), np.float32)
    assert sr.route(z, 3, "sigmoid", groups=4, kept=2, top=2)[0].tolist() == [[0, 1, 2]] * 3
    z[0, :7] = -np.inf
    ids, w = sr.route(z, 3, "softmax")
    assert ids[0].tolist() == [7, 0, 1] and w[0].tolist() == [1.0, 0.0, 0.0]
    z[:] = -np.inf
    ids, w = sr.route(z, 2, "softmax")
    assert ids.tolist() == [[0, 1]] * 3 and not w.any()


def test_int8_codes_by_brute_force():
    rng = np.random.default_rng(3)
    v = codecs.bf16_decode(codecs.bf16_encode(rng.standard_normal((5, 64)).astype(np.float32))).astype(np.float32)
    v[4] = 0
    c, s = int8.quantize_rows(v)
    assert np.abs(c[:4]).max(axis=1).tolist() == [127] * 4 and not c[4].any()
    grid = np.arange(-127, 128)
    for i in range(4):
        near = np.abs(v[i].astype(np.float64)[:, None] / float(s[i]) - grid[None, :])
        # the nearest code, up to the factor's rounding (2^-23 of 127)
        assert (np.take_along_axis(near, (c[i].astype(int) + 127)[:, None], 1)[:, 0] <= near.min(1) + 127 * 2.0 ** -22).all()
    w = rng.integers(-127, 128, (7, 64)).astype(np.int8)
    assert np.array_equal(int8.sums(c, w), c.astype(int) @ w.astype(int).T)


def test_int8_linear_is_the_formula():
    rng = np.random.default_rng(4)
    x = codecs.bf16_encode(rng.standard_normal((4, 48)).astype(np.float32))
    w = rng.integers(-127, 128, (9, 48)).astype(np.int8)
    s = rng.random(9).astype(np.float32)
    c, sx = int8.quantize_rows(codecs.bf16_decode(x))
    ref = (c.astype(np.float64) * sx[:, None]) @ (w.astype(np.float64) * s[:, None]).T
    assert np.allclose(int8.linear32(x, w, s), ref, rtol=4 * 2.0 ** -24, atol=1e-30)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("nxt", [True, False])
@pytest.mark.parametrize("k,shared,gated", [(3, True, True), (2, False, False), (0, True, False)])
def test_block_end_is_torchs(post, nxt, k, shared, gated):
    rng = np.random.default_rng(5)
    T, H = 4, 16
    leaf = {"y": rng.standard_normal((T * k, H)) if k else None, "w": rng.random((T, k)) if k else None,
            "shared": rng.standard_normal((T, H)) if shared else None, "gate": rng.random(T) if gated else None,
            "res": rng.standard_normal((T, H)), "post": rng.random(H) if post else None,
            "next": rng.random(H) if nxt else None}
    t = {n: torch.from_numpy(v).requires_grad_() if v is not None else None for n, v in leaf.items()}
    m = torch.zeros(T, H, dtype=torch.float64)
    if k:
        m = m + (t["w"][:, :, None] * t["y"].view(T, k, H)).sum(1)
    if shared:
        m = m + t["shared"] * (t["gate"][:, None] if gated else 1.0)
    if post:
        m = torch.nn.functional.rms_norm(m, (H,), t["post"], 1e-3)
    r = t["res"] + 0.5 * m
    a = [leaf[n] for n in ("y", "w", "shared", "gate")]
    ref, n, err = block_end.forward(*a, leaf["res"], leaf["post"], leaf["next"], 1e-3, 0.5)
    assert np.allclose(ref, r.detach().numpy(), rtol=1e-12) and (err >= np.abs(ref)).all()
    do, dn = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    loss = (r * torch.from_numpy(do)).sum()
    if nxt:
        h = torch.nn.functional.rms_norm(r, (H,), t["next"], 1e-3)
        assert np.allclose(n, h.detach().numpy(), rtol=1e-12)
        loss = loss + (h * torch.from_numpy(dn)).sum()
    loss.backward()
    got = block_end.backward(*a, ref, leaf["post"], leaf["next"], 1e-3, 0.5, do, dn if nxt else None)
    names = {"d_next": "next", "d_res": "res", "d_post": "post", "d_w": "w", "d_y": "y", "d_gate": "gate",
             "d_shared": "shared"}
    for g, at in names.items():
        assert (g in got) == (t[at] is not None)
        if g in got:
            v, mag = got[g]
            assert np.allclose(v, t[at].grad.numpy(), rtol=1e-10, atol=1e-13) and (mag >= np.abs(v) - 1e-13).all()
