"""One expert block as a program runs it: scored routing, permutation, experts on
8-bit weights, the block's end; and the training of its router: the end's gradients
into the routing's, on top of the losses'."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import block_end, codecs, int8, router as orouter, scored_routing as sr

pytestmark = pytest.mark.gpu
EPS, HALF, BF = 2.0 ** -24, 2.0 ** -8, torch.bfloat16


def _block(T, H, I, E, k, groups, seed):
    d = gh.dev()
    g = torch.Generator(device=d).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=d)  # noqa: E731
    w13, w2 = n(E, 2 * I, H) * H ** -0.5, n(E, H, I) * I ** -0.5
    s = {"x": n(T, H).to(BF), "logits": 2 * n(T, E), "bias": 0.1 * n(E), "shared": n(T, H).to(BF),
         "gate": torch.sigmoid(n(T)), "post": (1 + 0.1 * n(H)).to(BF), "next": (1 + 0.1 * n(H)).to(BF)}
    s["c13"], s["s13"] = torch.empty(E, 2 * I, H, dtype=torch.int8, device=d), torch.empty(E, 2 * I, device=d)
    s["c2"], s["s2"] = torch.empty(E, H, I, dtype=torch.int8, device=d), torch.empty(E, H, device=d)
    lib.moe_int8_quantize_weights(E, 2 * I, H, w13, s["c13"], s["s13"])
    lib.moe_int8_quantize_weights(E, H, I, w2, s["c2"], s["s2"])
    s["router"] = lib.make_router(E, k, "sigmoid", *groups, True, 2.5)
    s["shape"] = lib.make_shape(H, I, E, k, T, "bf16")
    i32 = dict(dtype=torch.int32, device=d)
    s.update(ids=torch.empty(T, k, **i32), w=torch.empty(T, k, device=d), off=torch.empty(E + 1, **i32),
             pairs=torch.empty(T * k, **i32), pos=torch.empty(T * k, **i32), y=torch.empty(T * k, H, dtype=BF, device=d),
             out=torch.empty(T, H, dtype=BF, device=d), normed=torch.empty(T, H, dtype=BF, device=d),
             ws=torch.empty(lib.moe_int8_experts_workspace_bytes(s["shape"]), dtype=torch.uint8, device=d))
    return s


def _run(s, T, H, k):
    lib.moe_route_scores(s["router"], T, s["logits"], s["ids"], s["w"], bias=s["bias"])
    lib.moe_permute(s["shape"], T, s["ids"], s["x"], s["off"], s["pairs"], s["pos"], s["x"])
    lib.moe_int8_experts(s["shape"], T, s["c13"], s["s13"], s["c2"], s["s2"], s["off"], s["pairs"], s["x"], s["y"], s["ws"])
    lib.moe_combine_norm(T, H, k, s["out"], s["normed"], y=s["y"], topk_w=s["w"], shared=s["shared"],
                         shared_gate=s["gate"], residual=s["x"], post_weight=s["post"], next_weight=s["next"], scale=0.5)


def _host(t):
    if t.dtype == BF:
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


@pytest.mark.parametrize("T", [1, 6, 70, 300])
def test_forward(T):
    H, I, E, k, groups = 256, 128, 16, 3, (4, 2, 2)
    s = _block(T, H, I, E, k, groups, T)
    _run(s, T, H, k)
    ids, w = sr.route(_host(s["logits"]), k, "sigmoid", _host(s["bias"]), *groups, True, 2.5)
    assert np.array_equal(_host(s["ids"]), ids)
    flat = ids.reshape(-1)
    off, pairs = np.r_[0, np.cumsum(np.bincount(flat, minlength=E))], np.argsort(flat, kind="stable")
    assert np.array_equal(_host(s["off"]), off) and np.array_equal(_host(s["pairs"]), pairs)
    y, _, _, _ = int8.experts(_host(s["x"]), *(_host(s[n]) for n in ("c13", "s13", "c2", "s2")), off, pairs, k)
    got = codecs.bf16_decode(_host(s["y"])).astype(np.float64)
    # rows whose intermediate meets a border between codes differ by code steps; over all rows that is little
    assert np.linalg.norm(got - y) <= HALF * np.linalg.norm(y)
    f = lambda n: s[n].double().cpu().numpy()  # noqa: E731
    r, n, err = block_end.forward(f("y"), f("w"), f("shared"), f("gate"), f("x"), f("post"), f("next"), 1e-6, 0.5)
    assert (np.abs(f("out") - r) <= HALF * np.abs(r) + 2 * EPS * err + 1e-40).all()
    assert (np.abs(f("normed") - n) <= HALF * np.abs(n) * 1.01 + 1e-5).all()


@pytest.mark.parametrize("T,seqs", [(5, 1), (200, 3)])
def test_router_training(T, seqs):
    """d_logits of the block's end and of the losses together, against the oracles chained in float64 (each stage's
    bounds as in its own tests, the losses' 32 roundings of their terms; the end's d_topk_w carries 180 2^-24 of its
    magnitude into the routing's)."""
    H, I, E, k, groups = 256, 128, 16, 3, (4, 2, 2)
    d = gh.dev()
    s = _block(T, H, I, E, k, groups, T + 7)
    _run(s, T, H, k)
    g = torch.Generator(device=d).manual_seed(3)
    d_out, d_normed = (torch.randn(T, H, generator=g, device=d).to(BF) for _ in range(2))
    d_w, d_y, d_res = torch.empty(T, k, device=d), torch.empty_like(s["y"]), torch.empty_like(d_out)
    dp, dn = torch.empty(H, device=d), torch.empty(H, device=d)
    ws = torch.empty(lib.moe_combine_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=d)
    lib.moe_combine_norm_backward(T, H, k, d_out, d_normed, s["out"], ws, y=s["y"], topk_w=s["w"], shared=s["shared"],
                                  shared_gate=s["gate"], post_weight=s["post"], next_weight=s["next"], scale=0.5,
                                  d_residual=d_res, d_y=d_y, d_topk_w=d_w, d_post_weight=dp, d_next_weight=dn)
    off = np.linspace(0, T, seqs + 1).astype(np.int32)
    offd = torch.from_numpy(off).to(d)
    loss, counts, tokens = torch.empty(2, device=d), torch.empty(seqs, E, dtype=torch.int32, device=d), torch.empty(seqs, dtype=torch.int32, device=d)
    bws = torch.empty(lib.moe_balance_loss_workspace_bytes(T, E, seqs), dtype=torch.uint8, device=d)
    lib.moe_balance_loss(T, E, k, s["logits"], s["ids"], loss, counts, tokens, bws, 0.5, 0.1, num_seqs=seqs, seq_offsets=offd)
    d_loss, d_logits = torch.ones(2, device=d), torch.empty(T, E, device=d)
    lib.moe_route_backward(T, E, k, s["logits"], s["ids"], d_logits, d_loss=d_loss, counts=counts, tokens=tokens,
                           balance_coef=0.5, z_coef=0.1, num_seqs=seqs, seq_offsets=offd)
    lib.moe_route_scores_backward(s["router"], T, s["logits"], s["ids"], d_w, d_logits, accumulate=True)
    f = lambda n: s[n].double().cpu().numpy()  # noqa: E731
    z, ids = _host(s["logits"]), _host(s["ids"])
    ref = block_end.backward(f("y"), f("w"), f("shared"), f("gate"), f("out"), f("post"), f("next"), 1e-6, 0.5,
                             d_out.double().cpu().numpy(), d_normed.double().cpu().numpy())
    rw, mw = ref["d_w"]
    a, ma = sr.backward(z, ids, rw, "sigmoid", True, 2.5)
    _, me = sr.backward(z, ids, mw, "sigmoid", True, 2.5)  # its magnitudes: what an error of d_topk_w becomes at most
    b, mb = orouter.backward(z, ids, d_loss=np.ones(2), coef=0.5, z_coef=0.1, seq_offsets=off)
    tol = EPS * (8 * ma + 180 * me + 32 * mb)
    bad = np.abs(d_logits.double().cpu().numpy() - (a + b)) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(d_logits.double().cpu().numpy() - (a + b))[bad][:4], tol[bad][:4])


def test_whole_block_captured():
    """The block in one graph, replayed on other inputs, against eager runs in between."""
    T, H, I, E, k = 48, 512, 256, 16, 4
    s = _block(T, H, I, E, k, (4, 2, 2), 1)
    _run(s, T, H, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(s, T, H, k)
    for i in range(3):
        s["x"].copy_(s["x"].flip(0).clone())
        s["logits"].mul_(-1.1)
        graph.replay()
        torch.cuda.synchronize()
        got = [s[n].clone() for n in ("ids", "w", "y", "out", "normed")]
        for n in ("ids", "w", "y", "out", "normed"):
            s[n].zero_()
        _run(s, T, H, k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, s[n]) for a, n in zip(got, ("ids", "w", "y", "out", "normed")))
