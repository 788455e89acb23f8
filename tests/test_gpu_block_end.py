"""The end of an expert block and its gradients against the float64 oracle.

Tolerances.  Forward: the oracle gives, beside r, what its fp32 roundings can be off
by in units of 2^-24 (k + 2 of the sum's magnitudes, 26 for a norm's factor: 46
additions of squares under a root, and 3 more); bf16 outputs add half a step, 2^-8 of the value.
normed multiplies r's error by its factor and adds the factor's own.  Gradients: every sum over a
row is of at most 16 values by a thread, 6 exchanges and 16 waves, with up to 20
roundings of a term before it: 60 per stage (next norm, sum and post norm, row sums),
180 2^-24 of the terms' magnitudes; the norm weights' sums over tokens add T / 512 in a
block, 32 of a wave's parts and 16 waves: 64 more for the sizes here."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import block_end, codecs

pytestmark = pytest.mark.gpu
EPS, HALF = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


def _inputs(T, H, k, shared, gate, post, nxt, res, seed=0):
    """Device tensors by name; None for what is absent."""
    d = gh.dev()
    g = torch.Generator(device=d).manual_seed(seed * 1000 + T + H + k)
    n = lambda *s: torch.randn(*s, generator=g, device=d)  # noqa: E731
    wide = 1.0 + 19.0 * (torch.rand(H, generator=g, device=d) < 0.02).float()
    return {"y": n(T * k, H).to(BF) if k else None, "topk_w": torch.softmax(n(T, k), 1) if k else None,
            "shared": n(T, H).to(BF) if shared else None, "shared_gate": torch.sigmoid(n(T)) if gate else None,
            "residual": (n(T, H) * wide).to(BF) if res else None,
            "post_weight": (1 + 0.3 * n(H)).to(BF) if post else None,
            "next_weight": (1 + 0.3 * n(H)).to(BF) if nxt else None,
            "out": (n(T, H) * wide).to(BF), "d_out": n(T, H).to(BF), "d_normed": n(T, H).to(BF) if nxt else None}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _forward(a, T, H, k, scale, eps):
    d = gh.dev()
    out = torch.full((T + 1, H), 7.0, dtype=BF, device=d)
    normed = torch.full((T + 1, H), 7.0, dtype=BF, device=d) if a["next_weight"] is not None else None
    names = ("y", "topk_w", "shared", "shared_gate", "residual", "post_weight", "next_weight")
    lib.moe_combine_norm(T, H, k, out, normed, scale=scale, eps=eps, **{n: a[n] for n in names})
    torch.cuda.synchronize()
    assert (out[T] == 7).all() and (normed is None or (normed[T] == 7).all())
    return out[:T], None if normed is None else normed[:T]


GRADS = {"d_residual": "d_res", "d_y": "d_y", "d_topk_w": "d_w", "d_shared": "d_shared", "d_gate": "d_gate",
         "d_post_weight": "d_post", "d_next_weight": "d_next"}


def _buffers(a, T, H, k):
    d = gh.dev()
    b = {"d_residual": torch.full((T + 1, H), 7.0, dtype=BF, device=d)}
    if k:
        b["d_y"], b["d_topk_w"] = torch.full((T * k + 1, H), 7.0, dtype=BF, device=d), torch.full((T + 1, k), 7.0, device=d)
    if a["shared"] is not None:
        b["d_shared"] = torch.full((T + 1, H), 7.0, dtype=BF, device=d)
    if a["shared_gate"] is not None:
        b["d_gate"] = torch.full((T + 1,), 7.0, device=d)
    for n in ("post_weight", "next_weight"):
        if a[n] is not None:
            b["d_" + n] = torch.full((H,), 7.0, device=d)
    return b


def _backward(a, T, H, k, scale, eps, b=None, ws=None):
    names = ("y", "topk_w", "shared", "shared_gate", "post_weight", "next_weight", "out", "d_normed")
    b = _buffers(a, T, H, k) if b is None else b
    if ws is None:
        ws = torch.full((lib.moe_combine_norm_backward_workspace_bytes(T, H),), 0xFF, dtype=torch.uint8, device=gh.dev())
    lib.moe_combine_norm_backward(T, H, k, a["d_out"], ws=ws, scale=scale, eps=eps, **{n: a[n] for n in names}, **b)
    return b


def _check(a, T, H, k, scale=0.5, eps=1e-5):
    p = {n: _np(v) for n, v in a.items()}
    out, normed = _forward(a, T, H, k, scale, eps)
    r, n, err = block_end.forward(p["y"], p["topk_w"], p["shared"], p["shared_gate"], p["residual"], p["post_weight"],
                                  p["next_weight"], eps, scale)
    tol = EPS * err
    assert (np.abs(_np(out) - r) <= HALF * np.abs(r) + (1 + HALF) * tol + 1e-40).all()
    if n is not None:
        q = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
        rel = 30 * EPS + q * np.sqrt((tol * tol).mean(1, keepdims=True))
        t32 = q * np.abs(p["next_weight"]) * tol + np.abs(n) * rel
        assert (np.abs(_np(normed) - n) <= HALF * np.abs(n) + (1 + HALF) * t32 + 1e-40).all()
    ref = block_end.backward(p["y"], p["topk_w"], p["shared"], p["shared_gate"], p["out"], p["post_weight"],
                             p["next_weight"], eps, scale, p["d_out"], p["d_normed"])
    b = _backward(a, T, H, k, scale, eps)
    torch.cuda.synchronize()
    for name, t in b.items():
        v, mag = ref[GRADS[name]]
        rows = len(v)
        if name not in ("d_post_weight", "d_next_weight"):
            assert (t[rows:] == 7).all()
        bound = (244 if rows == H and t.dim() == 1 and name != "d_gate" else 180) * EPS * mag
        if t.dtype == BF:
            bound = bound * (1 + HALF) + HALF * np.abs(v)
        bad = np.abs(_np(t)[:rows] - v) > bound + 1e-40
        assert not bad.any(), (name, np.argwhere(bad)[:4])


#        shared, gate, post, next, residual
FORMS = [(False, False, False, False, True), (True, False, False, True, True), (True, True, True, True, True),
         (False, False, True, False, True), (True, True, False, True, False), (False, False, True, True, False)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (3, 64, 2), (5, 520, 3), (2, 2048, 8), (7, 2056, 6), (33, 4096, 4),
                                   (3, 7168, 8), (2, 16384, 2), (600, 256, 2), (9, 1000, 9), (2, 128, 32), (4, 7176, 5)])
def test_sizes(T, H, k, form):
    _check(_inputs(T, H, k, *form), T, H, k)


@pytest.mark.parametrize("H,k", [(8, 3), (504, 10), (520, 12), (2056, 1), (8192, 8), (8200, 4), (16384, 32)])
def test_one_token(H, k):
    """The first launch alone has the norm weights' gradients then; they lie at any 4 bytes and end where they end."""
    a = _inputs(1, H, k, True, True, True, True, True)
    _check(a, 1, H, k)
    ref = _backward(a, 1, H, k, 0.5, 1e-5)
    b = _buffers(a, 1, H, k)
    hold = {n: torch.full((H + 5,), 7.0, device=gh.dev()) for n in ("d_post_weight", "d_next_weight")}
    for n, t in hold.items():
        b[n] = t[3:H + 3]
    _backward(a, 1, H, k, 0.5, 1e-5, b)
    torch.cuda.synchronize()
    assert all(torch.equal(b[n], ref[n]) for n in ref)
    assert all((t[:3] == 7).all() and (t[H + 3:] == 7).all() for t in hold.values())


@pytest.mark.parametrize("gate,post,nxt,res", [(False, False, True, False), (True, True, True, True), (False, True, False, True)])
@pytest.mark.parametrize("T,H", [(1, 8), (40, 1024), (6, 7168)])
def test_without_routed_experts(T, H, gate, post, nxt, res):
    _check(_inputs(T, H, 0, True, gate, post, nxt, res), T, H, 0, scale=1.0, eps=0.0)


def test_is_combine():
    """Without the other parts it is moe_combine, bit for bit."""
    a = _inputs(50, 1024, 6, False, False, False, False, False)
    out, _ = _forward(a, 50, 1024, 6, 1.0, 0.0)
    ref = torch.empty_like(out)
    lib.moe_combine(lib.make_shape(1024, 128, 8, 6, 50, "bf16"), 50, a["y"], a["topk_w"], ref)
    assert torch.equal(out, ref)


def test_in_place():
    a = _inputs(40, 2048, 4, True, True, True, True, True)
    out, normed = _forward(a, 40, 2048, 4, 0.5, 1e-5)
    names = ("y", "topk_w", "shared", "shared_gate", "post_weight", "next_weight")
    r, n = a["residual"].clone(), torch.empty_like(normed)
    lib.moe_combine_norm(40, 2048, 4, r, n, residual=r, scale=0.5, eps=1e-5, **{m: a[m] for m in names})
    assert torch.equal(r, out) and torch.equal(n, normed)
    b = _backward(a, 40, 2048, 4, 0.5, 1e-5)
    c = _buffers(a, 40, 2048, 4)
    a["d_out"] = c["d_residual"] = a["d_out"].clone()
    _backward(a, 40, 2048, 4, 0.5, 1e-5, c)
    assert torch.equal(c["d_residual"], b["d_residual"][:40]) and torch.equal(c["d_y"], b["d_y"])


def test_parts_that_are_not_wanted():
    """Each gradient alone is what it is among all; d_out may be absent."""
    a = _inputs(20, 512, 3, True, True, True, True, True)
    full = _backward(a, 20, 512, 3, 0.5, 1e-5)
    for name in ("d_residual", "d_y", "d_topk_w", "d_shared", "d_gate"):
        b = {n: v for n, v in _buffers(a, 20, 512, 3).items() if n == name or n.endswith("_weight")}
        _backward(a, 20, 512, 3, 0.5, 1e-5, b)
        assert all(torch.equal(b[n], full[n]) for n in b)
    a["d_out"] = torch.zeros_like(a["d_out"])
    zero = _backward(a, 20, 512, 3, 0.5, 1e-5)
    a["d_out"] = None
    none = _backward(a, 20, 512, 3, 0.5, 1e-5)
    assert all(torch.equal(zero[n], none[n]) for n in zero)


@pytest.mark.parametrize("T,k", [(30, 4), (1500, 2)])
def test_captured_and_on_another_stream(T, k):
    H, d = 1024, gh.dev()
    a = _inputs(T, H, k, True, True, True, True, True)
    fnames = ("y", "topk_w", "shared", "shared_gate", "residual", "post_weight", "next_weight")
    n = lib.moe_combine_norm_backward_workspace_bytes(T, H)
    ws = [torch.empty(n, dtype=torch.uint8, device=d) for _ in range(2)]
    o = [{**_buffers(a, T, H, k), "out": torch.zeros(T, H, dtype=BF, device=d), "normed": torch.zeros(T, H, dtype=BF, device=d)}
         for _ in range(2)]

    def step(i):
        lib.moe_combine_norm(T, H, k, o[i]["out"], o[i]["normed"], scale=0.5, eps=1e-5, **{m: a[m] for m in fnames})
        b = {m: v for m, v in o[i].items() if m not in ("out", "normed")}
        _backward({**a, "out": o[i]["out"]}, T, H, k, 0.5, 1e-5, b, ws[i])

    step(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(1)
    torch.cuda.synchronize()
    assert all(torch.equal(o[0][m], o[1][m]) for m in o[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(1)
    for i in range(3):
        a["y"].mul_(-1.5)
        a["d_out"].copy_(a["d_out"].flip(0).clone())
        for w in ws:
            w.fill_(0xFF)
        graph.replay()
        step(0)
        torch.cuda.synchronize()
        assert all(torch.equal(o[0][m], o[1][m]) for m in o[0])


def test_gradient_is_the_outputs_differences():
    """d(sum of out D + normed N) by a weight, a gate and a norm weight, from the oracle's float64 forward at inputs a
    step of 2^-10 apart (h^2 / 6 of the third derivative, which is below 4 of the loss's magnitude here), against the
    library's gradients at the forward's own rows: those are rounded to bf16, 2^-8 of each."""
    T, H, k, eps, scale, h = 3, 256, 2, 1e-3, 0.5, 2.0 ** -10
    a = _inputs(T, H, k, True, True, True, True, True)
    p = {n: _np(v) for n, v in a.items()}

    def loss(q):
        r, n, _ = block_end.forward(q["y"], q["topk_w"], q["shared"], q["shared_gate"], q["residual"], q["post_weight"],
                                    q["next_weight"], eps, scale)
        return (r * p["d_out"]).sum(1) + (n * p["d_normed"]).sum(1), (np.abs(r * p["d_out"])).sum(1) + np.abs(n * p["d_normed"]).sum(1)

    out, _ = _forward(a, T, H, k, scale, eps)
    b = _backward({**a, "out": out}, T, H, k, scale, eps)
    mag = loss(p)[1]
    for name, g in (("topk_w", "d_topk_w"), ("shared_gate", "d_gate")):
        for j in range(k if name == "topk_w" else 1):
            v = []
            for s in (h, -h):
                q = dict(p, **{name: p[name].copy()})
                if name == "topk_w":
                    q[name][:, j] += s
                else:
                    q[name] += s
                v.append(loss(q)[0])
            got = _np(b[g])[:T, j] if name == "topk_w" else _np(b[g])[:T]
            assert (np.abs((v[0] - v[1]) / (2 * h) - got) <= mag * (HALF + 4 * h * h / 6)).all()


def test_rows_that_are_not_finite():
    """A token with an infinity or a NaN says nothing about other tokens."""
    T, H, k = 30, 512, 3
    a = _inputs(T, H, k, True, True, True, True, True)
    out, normed = _forward(a, T, H, k, 0.5, 1e-5)
    b = _backward(a, T, H, k, 0.5, 1e-5)
    a["y"][4 * k + 1, 9], a["shared"][7, 100], a["topk_w"][9, 0] = float("nan"), float("inf"), float("nan")
    bad = torch.zeros(T, dtype=torch.bool, device=gh.dev())
    bad[[4, 7, 9]] = True
    out2, normed2 = _forward(a, T, H, k, 0.5, 1e-5)
    c = _backward(a, T, H, k, 0.5, 1e-5)
    assert torch.equal(out[~bad], out2[~bad]) and torch.equal(normed[~bad], normed2[~bad])
    assert torch.isnan(normed2[bad]).any(1).all()
    assert torch.equal(b["d_topk_w"][:T][~bad], c["d_topk_w"][:T][~bad])
    assert torch.equal(b["d_shared"][:T][~bad], c["d_shared"][:T][~bad])


def test_rows_past_2_31():
    """40000 tokens of 8 rows of 7168: 2.3e9 values; tokens at both ends."""
    T, H, k = 40000, 7168, 8
    a = _inputs(T, H, k, False, False, True, True, True)
    out, normed = _forward(a, T, H, k, 0.5, 1e-5)
    b = _backward(a, T, H, k, 0.5, 1e-5)
    for t in (0, 37449, 37450, T - 1):
        s = {n: None if v is None else v if n.endswith("_weight") else v[t * k:(t + 1) * k] if n == "y" else v[t:t + 1]
             for n, v in a.items()}
        o, n = _forward(s, 1, H, k, 0.5, 1e-5)
        g = _backward(s, 1, H, k, 0.5, 1e-5)
        assert torch.equal(o[0], out[t]) and torch.equal(n[0], normed[t])
        assert torch.equal(g["d_y"][:k], b["d_y"][t * k:(t + 1) * k]) and torch.equal(g["d_topk_w"][0], b["d_topk_w"][t])
