"""Host-side refusals of the block-128 fp8 products and the router's training
operators (no GPU is touched: nothing is enqueued), and their sizes."""
import ctypes

import pytest

import mixture_experts_layer_sort_amd as lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
A = 1 << 20  # an address that is never read


def up(n):
    return (n + 255) // 256 * 256


def linear(**kw):
    a = dict(M=2, N=256, K=256, codes=A, scales=A, x=A, xs=256, out=A, os=256, ws=A, nbytes=1 << 30)
    a.update(kw)
    return lib.load().moe_fp8_linear(a["M"], a["N"], a["K"], a["codes"], a["scales"], a["x"], a["xs"], a["out"],
                                     a["os"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", [
    ({"N": 0}, UNSUPPORTED), ({"N": (1 << 20) + 1}, UNSUPPORTED), ({"K": 0}, UNSUPPORTED), ({"K": 8}, UNSUPPORTED),
    ({"K": 264}, UNSUPPORTED), ({"K": (1 << 20) + 16}, UNSUPPORTED), ({"M": -1}, INVALID),
    ({"M": (1 << 24) + 1}, INVALID), ({"M": 0, "codes": None}, OK),
    ({"codes": None}, INVALID), ({"scales": None}, INVALID), ({"x": None}, INVALID), ({"out": None}, INVALID),
    ({"ws": None}, INVALID), ({"codes": A + 8}, INVALID), ({"x": A + 8}, INVALID), ({"scales": A + 2}, INVALID),
    ({"out": A + 1}, INVALID), ({"ws": A + 16}, INVALID), ({"xs": 255}, INVALID), ({"xs": 260}, INVALID),
    ({"xs": -256}, INVALID), ({"os": 255}, INVALID), ({"xs": (1 << 32) + 8}, UNSUPPORTED),
    ({"os": (1 << 32) + 1}, UNSUPPORTED), ({"nbytes": 64}, WORKSPACE),
])
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


def test_linear_workspace():
    f = lib.moe_fp8_linear_workspace_bytes
    assert f(5, 100, 272) == up(5 * 384) + up(5 * 3 * 4)
    assert f(0, 100, 256) == 0 and f(5, 0, 256) == 0 and f(5, 100, 250) == 0 and f((1 << 24) + 1, 1, 16) == 0


def test_quantize_weights_refusals():
    f = lib.load().moe_fp8_quantize_weights
    assert f(1, 4, 24, A, A, A, None) == UNSUPPORTED and f(1, 0, 32, A, A, A, None) == UNSUPPORTED
    assert f(-1, 4, 32, A, A, A, None) == INVALID and f(0, 4, 32, None, None, None, None) == OK
    assert f(1, 4, 32, None, A, A, None) == INVALID and f(1, 4, 32, A + 4, A, A, None) == INVALID
    assert f(1 << 30, 256, 256, A, A, A, None) == UNSUPPORTED


def experts(shape=None, **kw):
    a = dict(T=2, w13=A, s13=A, w2=A, s2=A, off=A, pairs=A, x=A, y=A, ws=A, nbytes=1 << 40)
    a.update(kw)
    s = shape if shape is not None else lib.make_shape(256, 128, 8, 2, 16, "bf16")
    return lib.load().moe_fp8_experts(ctypes.byref(s), a["T"], a["w13"], a["s13"], a["w2"], a["s2"], a["off"],
                                      a["pairs"], a["x"], a["y"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"T": 17}, INVALID), ({"T": 0, "w13": None}, OK), ({"w13": None}, INVALID),
    ({"s13": None}, INVALID), ({"w2": None}, INVALID), ({"s2": None}, INVALID), ({"off": None}, INVALID),
    ({"pairs": None}, INVALID), ({"x": None}, INVALID), ({"y": None}, INVALID), ({"ws": None}, INVALID),
    ({"w2": A + 8}, INVALID), ({"x": A + 2}, INVALID), ({"y": A + 4}, INVALID), ({"ws": A + 128}, INVALID),
    ({"nbytes": 64}, WORKSPACE),
])
def test_experts_refusals(kw, status):
    assert experts(**kw) == status


def test_experts_shapes():
    for dt in ("mxfp8", "nvfp4", "bf16_mxfp8"):
        s = lib.make_shape(256, 128, 8, 2, 16, dt)
        assert experts(s) == UNSUPPORTED and lib.moe_fp8_experts_workspace_bytes(s) == 0
    assert experts(lib.make_shape(256, 128, 8, 2, 16, "bf16", "relu2")) == UNSUPPORTED
    assert experts(lib.make_shape(200, 128, 8, 2, 16, "bf16")) == UNSUPPORTED
    assert experts(lib.make_shape(256, 128, 8, 2, 16, "bf16", gate_up_limit=-1.0)) == INVALID
    assert lib.load().moe_fp8_experts(None, 1, A, A, A, A, A, A, A, A, A, 1 << 40, None) == INVALID
    assert lib.moe_fp8_experts_workspace_bytes(lib.make_shape(256, 128, 8, 2, 16, "bf16")) > 0


def balance(**kw):
    a = dict(T=4, E=8, k=2, logits=A, ids=A, mask=None, S=1, seq=None, c=0.1, z=0.1, loss=A, counts=A, tokens=A, ws=A,
             nbytes=1 << 30)
    a.update(kw)
    return lib.load().moe_balance_loss(a["T"], a["E"], a["k"], a["logits"], a["ids"], a["mask"], a["S"], a["seq"],
                                       a["c"], a["z"], a["loss"], a["counts"], a["tokens"], a["ws"], a["nbytes"], None)


def backward(**kw):
    a = dict(T=4, E=8, k=2, logits=A, ids=A, w=A, dw=A, mask=None, S=1, seq=None, c=0.1, z=0.1, counts=A, tokens=A,
             dl=A, out=A)
    a.update(kw)
    return lib.load().moe_route_backward(a["T"], a["E"], a["k"], a["logits"], a["ids"], a["w"], a["dw"], a["mask"],
                                         a["S"], a["seq"], a["c"], a["z"], a["counts"], a["tokens"], a["dl"],
                                         a["out"], None)


@pytest.mark.parametrize("call", [balance, backward])
@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"T": 0, "logits": None}, OK), ({"E": 0}, UNSUPPORTED), ({"E": 1025}, UNSUPPORTED),
    ({"k": 0}, UNSUPPORTED), ({"k": 9}, UNSUPPORTED), ({"E": 64, "k": 33}, UNSUPPORTED),
    ({"T": (1 << 23) + 1}, UNSUPPORTED), ({"S": 0}, INVALID), ({"S": 2}, INVALID), ({"S": 65537, "seq": A}, UNSUPPORTED),
    ({"c": float("nan")}, INVALID), ({"z": float("inf")}, INVALID), ({"logits": None}, INVALID), ({"counts": None}, INVALID),
    ({"tokens": None}, INVALID), ({"ids": None}, INVALID),
])
def test_router_refusals(call, kw, status):
    assert call(**kw) == status


def test_router_refusals_of_one_side():
    assert balance(loss=None) == INVALID and balance(ws=None) == INVALID and balance(ws=A + 64) == INVALID
    assert balance(nbytes=64) == WORKSPACE
    assert backward(out=None) == INVALID and backward(w=None) == INVALID
    assert backward(dw=None, dl=None) == INVALID
    f = lib.moe_balance_loss_workspace_bytes
    assert f(0, 8, 1) == 0 and f(4, 1025, 1) == 0 and f(4, 8, 0) == 0 and f(4, 8, 1) > 0
    assert f((1 << 24) + 1, 8, 1) == 0 and f(4, 8, 65537) == 0


def test_workspace_of_a_large_batch_serves_smaller_ones():
    """Sizes never fall as a batch grows: across 16384 tokens, where chunks begin to grow, and at each later step."""
    f = lib.moe_balance_loss_workspace_bytes
    tokens = sorted({t + d for t in (1, 16, 128, 1000, *range(16384, 70000, 1024), 1 << 20, 1 << 24) for d in (-1, 0, 1)})
    tokens = [t for t in tokens if 1 <= t <= 1 << 24]
    for E, S in ((1, 1), (256, 16), (1024, 40)):
        sizes = [f(t, E, S) for t in tokens]
        assert sizes == sorted(sizes), (E, S)
    assert f(5000, 64, 1) <= f(5000, 64, 2) <= f(5000, 64, 1000) <= f(5000, 64, 65536)
    assert f(5000, 1, 3) <= f(5000, 64, 3) <= f(5000, 65, 3) <= f(5000, 1024, 3)
    assert balance(T=16384, E=256, S=16, seq=A, nbytes=f(16384, 256, 16) - 1) == WORKSPACE


@pytest.mark.parametrize("name", ["s13", "s2", "off", "pairs"])
def test_experts_refuse_odd_addresses(name):
    assert experts(**{name: A + 2}) == INVALID and experts(**{name: A + 1}) == INVALID


@pytest.mark.parametrize("call,names", [
    (balance, ("logits", "ids", "seq", "loss", "counts", "tokens")),
    (backward, ("logits", "ids", "w", "dw", "seq", "counts", "tokens", "dl", "out")),
])
def test_router_refuses_odd_addresses(call, names):
    for name in names:
        assert call(**{"seq": A, name: A + 2}) == INVALID, name


def test_quantize_weights_refuses_more_blocks_than_a_launch_has():
    """A launch has fewer than 2^32 threads, and a block of 128 x 128 weights takes 256."""
    f = lib.load().moe_fp8_quantize_weights
    assert f(1 << 24, 1, 16, A, A, A, None) == UNSUPPORTED and f(1 << 22, 129, 144, A, A, A, None) == UNSUPPORTED
    assert f((1 << 24) - 1, 1, 16, None, A, A, None) == INVALID
