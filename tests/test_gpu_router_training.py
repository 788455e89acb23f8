"""Balance loss, counts and the router's gradient against the float64 oracle.

Tolerances.  A probability: the exponent's argument (below 2^6 in magnitude)
is rounded twice at 2^-24 relative, exp and the quotient at a few 2^-24: 2^-17
relative is more than their sum.  Gradients are held to 2^-17 of the sum of the
magnitudes of their terms, the losses (long sums of such probabilities, of
which errors average) to 2^-17 relative.  Counts are whole numbers: equal."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import router

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -17


def _case(T, E, k, S, masked, seed=0):
    rng = np.random.default_rng(seed + T * 31 + E)
    logits = (rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)).astype(np.float32)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    off = np.sort(np.concatenate([[0, T], rng.integers(0, T + 1, S - 1)])).astype(np.int32)
    mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
    if masked and S > 1:
        mask[off[1]:off[2]] = 0  # a sequence of padding only
    return rng, logits, ids, off, mask


def _dev(v):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(gh.dev())


def _loss(logits, ids, off, mask, coef, z):
    T, E = logits.shape
    S, d = len(off) - 1, gh.dev()
    loss = torch.full((2,), 9.0, device=d)
    counts = torch.full((S, E), -1, dtype=torch.int32, device=d)
    tokens = torch.full((S,), -1, dtype=torch.int32, device=d)
    ws = torch.full((lib.moe_balance_loss_workspace_bytes(T, E, S),), 0xFF, dtype=torch.uint8, device=d)
    lib.moe_balance_loss(T, E, ids.shape[1], _dev(logits), _dev(ids), loss, counts, tokens, ws, coef, z,
                         token_mask=_dev(mask), num_seqs=S, seq_offsets=_dev(off))
    torch.cuda.synchronize()
    return loss, counts, tokens


def _grad(logits, ids, off, mask, coef, z, w=None, dw=None, dl=None, counts=None, tokens=None):
    T, E = logits.shape
    out = torch.full((T + 1, E), 9.0, device=gh.dev())
    lib.moe_route_backward(T, E, ids.shape[1], _dev(logits), _dev(ids), out, topk_w=_dev(w), d_topk_w=_dev(dw),
                           d_loss=_dev(dl), counts=counts, tokens=tokens, balance_coef=coef, z_coef=z,
                           token_mask=_dev(mask), num_seqs=len(off) - 1, seq_offsets=_dev(off))
    torch.cuda.synchronize()
    assert bool((out[T] == 9.0).all())
    return out[:T].double().cpu().numpy()


CASES = [  # T, E, k, sequences, masked
    (1, 1, 1, 1, False), (1, 5, 2, 1, False), (1, 256, 8, 1, False), (7, 64, 6, 1, True), (63, 65, 1, 2, False),
    (64, 128, 8, 4, True), (100, 132, 4, 3, True), (200, 256, 8, 16, False), (333, 260, 10, 5, True),
    (129, 384, 8, 2, False), (50, 512, 8, 1, True), (77, 600, 32, 3, False), (40, 1024, 32, 2, True),
    (33, 1023, 3, 2, True), (2500, 12, 2, 40, True), (20000, 16, 2, 3, False),
]


@pytest.mark.parametrize("T,E,k,S,masked", CASES)
def test_loss_and_gradient(T, E, k, S, masked):
    rng, logits, ids, off, mask = _case(T, E, k, S, masked)
    loss, counts, tokens = _loss(logits, ids, off, mask, 0.01, 0.001)
    rl, rc, rt = router.balance_loss(logits, ids, 0.01, 0.001, mask, off)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    got = loss.double().cpu().numpy()
    print(f"  T={T} E={E}: loss {got} rel {np.abs(got - rl) / np.maximum(np.abs(rl), 1e-30)}", flush=True)
    assert np.all(np.abs(got - rl) <= TOL * np.abs(rl))
    w = np.take_along_axis(logits, ids, 1)
    w = (np.exp(w - w.max(1, keepdims=True)) / np.exp(w - w.max(1, keepdims=True)).sum(1, keepdims=True)).astype(np.float32)
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    dl = np.array([1.5, -0.5], np.float32)
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        a = (w, dw) if use_w else (None, None)
        l = dl if use_l else None
        ref, mag = router.backward(logits, ids, *a, l, 0.01, 0.001, mask, off)
        g = _grad(logits, ids, off, mask, 0.01, 0.001, *a, l, counts if use_l else None, tokens if use_l else None)
        bad = np.abs(g - ref) > TOL * mag
        assert not bad.any(), (use_w, use_l, np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4])
    if mask is not None:
        assert not g[mask == 0].any()


def test_gradient_is_the_losses_differences():
    """Central differences of the loss that the library itself computes.  The loss is an fp32 number (2^-24
    relative) and the step 2^-3: differences are off by 2^-24 L / 2^-3 from rounding and by h^2 / 6 of the
    third derivative, which for a softmax is below the loss's scale."""
    rng, logits, ids, off, mask = _case(6, 8, 2, 2, False, 3)
    coef, z, h = 1.0, 0.0, 0.125
    loss, counts, tokens = _loss(logits, ids, off, mask, coef, z)
    g = _grad(logits, ids, off, mask, coef, z, None, None, np.array([1.0, 0.0], np.float32), counts, tokens)
    L = float(loss[0])
    for t in range(6):
        for e in range(8):
            v = []
            for sgn in (1, -1):
                m = logits.copy()
                m[t, e] += sgn * h
                v.append(float(_loss(m, ids, off, mask, coef, z)[0][0]))
            assert abs((v[0] - v[1]) / (2 * h) - g[t, e]) <= 2.0 ** -20 * L + h * h / 6 * L


def test_masked_tokens_are_not_read():
    rng, logits, ids, off, mask = _case(90, 256, 4, 3, True, 4)
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    w = np.full(ids.shape, 0.25, np.float32)
    dl = np.array([1.0, 1.0], np.float32)
    a = _loss(logits, ids, off, mask, 0.1, 0.1)
    ga = _grad(logits, ids, off, mask, 0.1, 0.1, w, dw, dl, a[1], a[2])
    gone = mask == 0
    logits[gone], ids[gone], dw[gone], w[gone] = np.nan, 1 << 30, np.inf, np.nan
    b = _loss(logits, ids, off, mask, 0.1, 0.1)
    gb = _grad(logits, ids, off, mask, 0.1, 0.1, w, dw, dl, a[1], a[2])
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and np.array_equal(ga, gb)


def test_nothing_valid():
    _, logits, ids, off, _ = _case(40, 64, 4, 3, False, 5)
    mask = np.zeros(40, np.uint8)
    loss, counts, tokens = _loss(logits, ids, off, mask, 0.1, 0.1)
    assert not loss.any() and not counts.any() and not tokens.any()
    g = _grad(logits, ids, off, mask, 0.1, 0.1, None, None, np.ones(2, np.float32), counts, tokens)
    assert not g.any()


@pytest.mark.parametrize("T", [30, 400])
def test_logits_at_the_ends_of_the_type(T):
    """Rows of only the lowest value, only the largest, and both: no overflow.  (Without the z-loss, whose square is
    beyond fp32 there.)  Probabilities are 1 / E, 0 or 1 with the usual roundings."""
    rng, logits, ids, off, mask = _case(T, 96, 3, 2, True, 12)
    top, low = np.finfo(np.float32).max, np.finfo(np.float32).min
    logits[1::7] = low
    logits[2::7] = top
    logits[3::7] = low
    logits[3::7, 50] = top
    loss, counts, tokens = _loss(logits, ids, off, mask, 0.5, 0.0)
    rl, rc, rt = router.balance_loss(logits, ids, 0.5, 0.0, mask, off)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    assert rl[1] == 0 and float(loss[1]) == 0
    assert abs(float(loss[0]) - rl[0]) <= TOL * abs(rl[0])
    w = rng.random(ids.shape).astype(np.float32)
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    ref, mag = router.backward(logits, ids, w, dw, (1.0, 1.0), 0.5, 0.0, mask, off)
    g = _grad(logits, ids, off, mask, 0.5, 0.0, w, dw, np.ones(2, np.float32), counts, tokens)
    bad = np.abs(g - ref) > 4 * TOL * mag + 2.0 ** -123
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4], mag[bad][:4])


def test_switched_off_experts_extreme_logits_and_odd_ids():
    """-inf logits and the type's lowest value have probability zero; ids outside are not counted, an id twice is.
    Row 0's exponents reach -87: the difference is rounded at 2^6 2^-24 = 2^-18, its product with log2 e (up to 2^7)
    twice at 2^7 2^-24 ln 2, together 1.6e-5 relative, held to 2^-15; and a probability below 2^-126,
    fp32's smallest normal number, may be taken for zero: times its factor |A| + sum p |A| + |Z lse|, at most 2 from
    the z-loss (0.25 * 2 * 80 / (2 n), n >= 10) and 4 from the balance loss (0.5 / (2 n) * E / k twice), an absolute
    2^3 2^-126 beside it."""
    rng, logits, ids, off, mask = _case(30, 200, 4, 2, True, 6)
    logits[:, 3] = -np.inf
    logits[:, 4] = np.finfo(np.float32).min
    logits[0, 7] = 80.0
    ids[ids == 3] = 5
    ids[ids == 4] = 5
    ids[2] = [-1, 200, 9, 9]
    loss, counts, tokens = _loss(logits, ids, off, mask, 0.5, 0.25)
    rl, rc, rt = router.balance_loss(logits, ids, 0.5, 0.25, mask, off)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= TOL * np.abs(rl))
    w = rng.random(ids.shape).astype(np.float32)
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    ref, mag = router.backward(logits, ids, w, dw, (1.0, 1.0), 0.5, 0.25, mask, off)
    g = _grad(logits, ids, off, mask, 0.5, 0.25, w, dw, np.ones(2, np.float32), counts, tokens)
    bad = np.abs(g - ref) > 4 * TOL * mag + 2.0 ** -123
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4], mag[bad][:4])


def test_tokens_in_no_sequence():
    """Offsets that begin after the first token and end before the last one."""
    rng, logits, ids, _, mask = _case(50, 64, 4, 1, True, 7)
    off = np.array([9, 9, 30, 41], np.int32)
    loss, counts, tokens = _loss(logits, ids, off, mask, 0.5, 0.25)
    rl, rc, rt = router.balance_loss(logits, ids, 0.5, 0.25, mask, off)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= TOL * np.abs(rl))
    w, dw = rng.random(ids.shape).astype(np.float32), rng.standard_normal(ids.shape).astype(np.float32)
    ref, mag = router.backward(logits, ids, w, dw, (1.0, 1.0), 0.5, 0.25, mask, off)
    g = _grad(logits, ids, off, mask, 0.5, 0.25, w, dw, np.ones(2, np.float32), counts, tokens)
    assert np.all(np.abs(g - ref) <= TOL * mag)


@pytest.mark.parametrize("T", [128, 129, 3000])
def test_tokens_outside_of_many_sequences(T):
    """Empty sequences, some of one token, tokens before the first and behind the last, around the sizes where the
    number of launches changes."""
    rng, logits, ids, _, mask = _case(T, 60, 3, 1, True, 17)
    off = np.array([5, 5, 6, 7, 7, T // 2, T // 2 + 1, T - 20, T - 20], np.int32)
    loss, counts, tokens = _loss(logits, ids, off, mask, 0.5, 0.25)
    rl, rc, rt = router.balance_loss(logits, ids, 0.5, 0.25, mask, off)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(tokens.cpu().numpy(), rt)
    assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= TOL * np.abs(rl))
    again = _loss(logits, ids, off, mask, 0.5, 0.25)
    assert torch.equal(again[0], loss)
    w, dw = rng.random(ids.shape).astype(np.float32), rng.standard_normal(ids.shape).astype(np.float32)
    ref, mag = router.backward(logits, ids, w, dw, (1.0, 1.0), 0.5, 0.25, mask, off)
    g = _grad(logits, ids, off, mask, 0.5, 0.25, w, dw, np.ones(2, np.float32), counts, tokens)
    assert np.all(np.abs(g - ref) <= TOL * mag)


def test_unaligned_rows_and_one_sequence_without_offsets():
    """Logits and gradients that begin 4 bytes into an allocation (no 16-byte rows), offsets left out."""
    rng, logits, ids, off, _ = _case(37, 256, 8, 1, False, 8)
    d = gh.dev()
    T, E, k = 37, 256, 8
    flat = torch.empty(T * E + 1, device=d)
    flat[1:] = _dev(logits).reshape(-1)
    loss, counts, tokens = torch.empty(2, device=d), torch.empty(1, E, dtype=torch.int32, device=d), torch.empty(1, dtype=torch.int32, device=d)
    ws = torch.empty(lib.moe_balance_loss_workspace_bytes(T, E), dtype=torch.uint8, device=d)
    lib.moe_balance_loss(T, E, k, flat[1:], _dev(ids), loss, counts, tokens, ws, 0.5, 0.25)
    rl, rc, _ = router.balance_loss(logits, ids, 0.5, 0.25)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= TOL * np.abs(rl))
    out = torch.empty(T * E + 1, device=d)
    lib.moe_route_backward(T, E, k, flat[1:], _dev(ids), out[1:], d_loss=torch.ones(2, device=d), counts=counts,
                           tokens=tokens, balance_coef=0.5, z_coef=0.25)
    ref, mag = router.backward(logits, ids, None, None, (1.0, 1.0), 0.5, 0.25)
    assert np.all(np.abs(out[1:].view(T, E).double().cpu().numpy() - ref) <= TOL * mag)


def test_router_step_captured():
    """route, loss and gradient in one graph, replayed with other logits beside eager runs; every replay equal to
    the eager results bit for bit."""
    d, (T, E, k) = gh.dev(), (700, 256, 8)
    shape = lib.make_shape(256, 128, E, k, T, "bf16")
    logits = torch.empty(T, E, device=d)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=d), torch.empty(T, k, device=d)
    ws = torch.empty(lib.moe_balance_loss_workspace_bytes(T, E, 2), dtype=torch.uint8, device=d)
    off = torch.tensor([0, 300, T], dtype=torch.int32, device=d)
    dw, dl = torch.randn(T, k, device=d), torch.ones(2, device=d)

    def step(out):
        lib.moe_route(shape, T, logits, ids, w)
        lib.moe_balance_loss(T, E, k, logits, ids, out[0], out[1], out[2], ws, 0.01, 0.001, num_seqs=2, seq_offsets=off)
        lib.moe_route_backward(T, E, k, logits, ids, out[3], topk_w=w, d_topk_w=dw, d_loss=dl, counts=out[1],
                               tokens=out[2], balance_coef=0.01, z_coef=0.001, num_seqs=2, seq_offsets=off)

    def outs():
        return (torch.empty(2, device=d), torch.empty(2, E, dtype=torch.int32, device=d),
                torch.empty(2, dtype=torch.int32, device=d), torch.empty(T, E, device=d))

    a, b = outs(), outs()
    logits.normal_()
    step(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    for _ in range(4):
        logits.normal_()
        g.replay()
        torch.cuda.synchronize()
        step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b))
