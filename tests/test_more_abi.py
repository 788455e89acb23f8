"""Host-side refusals of the scored routing, the 8-bit integer products and the end
of an expert block (no GPU is touched: nothing is enqueued), and their sizes."""
import ctypes

import pytest

import mixture_experts_layer_sort_amd as lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
A = 1 << 20  # an address that is never read


def up(n):
    return (n + 255) // 256 * 256


def router(E=64, k=4, score="sigmoid", **kw):
    return lib.make_router(E, k, score, **kw)


def route(r=None, **kw):
    a = dict(T=2, logits=A, ld=64, bias=A, ids=A, w=A)
    a.update(kw)
    r = r if r is not None else router()
    return lib.load().moe_route_scores(ctypes.byref(r), a["T"], a["logits"], a["ld"], a["bias"], a["ids"], a["w"], None)


ROUTERS = [
    (dict(E=0), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(k=0), UNSUPPORTED), (dict(k=33), UNSUPPORTED),
    (dict(E=3, k=4), UNSUPPORTED), (dict(score=2), UNSUPPORTED), (dict(score=-1), UNSUPPORTED),
    (dict(num_groups=0), UNSUPPORTED), (dict(num_groups=7), UNSUPPORTED), (dict(num_groups=128), UNSUPPORTED),
    (dict(num_groups=8, topk_groups=0), UNSUPPORTED), (dict(num_groups=8, topk_groups=9), UNSUPPORTED),
    (dict(num_groups=32, topk_groups=1), UNSUPPORTED),  # two experts for four picks
    (dict(num_groups=8, topk_groups=4, group_top=3), UNSUPPORTED), (dict(group_top=0), UNSUPPORTED),
    (dict(num_groups=64, topk_groups=8, group_top=2), UNSUPPORTED),
    (dict(renormalise=2), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
]


@pytest.mark.parametrize("kw,status", ROUTERS)
def test_router_refusals(kw, status):
    assert route(router(**kw)) == status
    r = router(**kw)
    assert lib.load().moe_route_scores_backward(ctypes.byref(r), 2, A, 64, A, A, None, 0, A, 64, None) == status


@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"T": 0, "logits": None}, OK), ({"logits": None}, INVALID), ({"ids": None}, INVALID),
    ({"w": None}, INVALID), ({"logits": A + 2}, INVALID), ({"bias": A + 1}, INVALID), ({"ids": A + 2}, INVALID),
    ({"w": A + 3}, INVALID), ({"ld": 63}, INVALID), ({"ld": -64}, INVALID), ({"ld": (1 << 32) + 1}, UNSUPPORTED),
    ({"T": (1 << 22) + 1}, UNSUPPORTED),
])
def test_route_refusals(kw, status):
    assert route(**kw) == status
    assert lib.load().moe_route_scores(None, 2, A, 64, A, A, A, None) == INVALID


def test_route_backward_refusals():
    f, r = lib.load().moe_route_scores_backward, router()
    p = ctypes.byref(r)
    assert f(None, 2, A, 64, A, A, None, 0, A, 64, None) == INVALID
    assert f(p, 0, None, 64, None, None, None, 0, None, 64, None) == OK
    assert f(p, -1, A, 64, A, A, None, 0, A, 64, None) == INVALID
    for i in (2, 4, 5, 8):
        a = [p, 2, A, 64, A, A, None, 0, A, 64, None]
        a[i] = None
        assert f(*a) == INVALID
        a[i] = A + 2
        assert f(*a) == INVALID
    assert f(p, 2, A, 63, A, A, None, 0, A, 64, None) == INVALID
    assert f(p, 2, A, 64, A, A, None, 0, A, 63, None) == INVALID
    assert f(p, 2, A, 64, A, A, None, 2, A, 64, None) == INVALID
    assert f(p, 2, A, 64, A, A, None, 0, A, (1 << 32) + 1, None) == UNSUPPORTED
    assert f(p, (1 << 22) + 1, A, 64, A, A, None, 0, A, 64, None) == UNSUPPORTED


def linear(**kw):
    a = dict(M=2, N=256, K=256, codes=A, scales=A, x=A, xs=256, out=A, os=256, ws=A, nbytes=1 << 30)
    a.update(kw)
    return lib.load().moe_int8_linear(a["M"], a["N"], a["K"], a["codes"], a["scales"], a["x"], a["xs"], a["out"],
                                      a["os"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", [
    ({"N": 0}, UNSUPPORTED), ({"N": (1 << 20) + 1}, UNSUPPORTED), ({"K": 0}, UNSUPPORTED), ({"K": 8}, UNSUPPORTED),
    ({"K": 264}, UNSUPPORTED), ({"K": (1 << 17) + 16}, UNSUPPORTED), ({"M": -1}, INVALID),
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
    f = lib.moe_int8_linear_workspace_bytes
    assert f(0, 100, 256) == 0 and f(5, 0, 256) == 0 and f(5, 100, 250) == 0 and f((1 << 24) + 1, 1, 16) == 0
    assert f(5, 100, (1 << 17) + 16) == 0
    for N, K in ((100, 272), (2816, 4096), (576, 7168), (64, 1 << 17)):
        sizes = [f(M, N, K) for M in (1, 2, 8, 16, 17, 32, 33, 64, 65, 128, 129, 500, 4096)]
        assert sizes == sorted(sizes) and sizes[0] > 0, (N, K)  # those of the largest serve all


def test_quantize_weights_refusals():
    f = lib.load().moe_int8_quantize_weights
    assert f(1, 4, 24, A, A, A, None) == UNSUPPORTED and f(1, 0, 32, A, A, A, None) == UNSUPPORTED
    assert f(-1, 4, 32, A, A, A, None) == INVALID and f(0, 4, 32, None, None, None, None) == OK
    assert f(1, 4, 32, None, A, A, None) == INVALID and f(1, 4, 32, A + 4, A, A, None) == INVALID
    assert f(1, 4, 32, A, A + 2, A, None) == INVALID and f(1, 4, 32, A, A, A + 1, None) == INVALID
    assert f(16, 1 << 20, 256, A, A, A, None) == UNSUPPORTED


def experts(shape=None, **kw):
    a = dict(T=2, w13=A, s13=A, w2=A, s2=A, off=A, pairs=A, x=A, y=A, ws=A, nbytes=1 << 40)
    a.update(kw)
    s = shape if shape is not None else lib.make_shape(256, 128, 8, 2, 16, "bf16")
    return lib.load().moe_int8_experts(ctypes.byref(s), a["T"], a["w13"], a["s13"], a["w2"], a["s2"], a["off"],
                                       a["pairs"], a["x"], a["y"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"T": 17}, INVALID), ({"T": 0, "w13": None}, OK), ({"w13": None}, INVALID),
    ({"s13": None}, INVALID), ({"w2": None}, INVALID), ({"s2": None}, INVALID), ({"off": None}, INVALID),
    ({"pairs": None}, INVALID), ({"x": None}, INVALID), ({"y": None}, INVALID), ({"ws": None}, INVALID),
    ({"w2": A + 8}, INVALID), ({"x": A + 2}, INVALID), ({"y": A + 4}, INVALID), ({"ws": A + 128}, INVALID),
    ({"s13": A + 2}, INVALID), ({"s2": A + 1}, INVALID), ({"off": A + 2}, INVALID), ({"pairs": A + 2}, INVALID),
    ({"nbytes": 64}, WORKSPACE),
])
def test_experts_refusals(kw, status):
    assert experts(**kw) == status


def test_experts_shapes():
    for dt in ("mxfp8", "nvfp4", "bf16_mxfp8"):
        s = lib.make_shape(256, 128, 8, 2, 16, dt)
        assert experts(s) == UNSUPPORTED and lib.moe_int8_experts_workspace_bytes(s) == 0
    assert experts(lib.make_shape(256, 128, 8, 2, 16, "bf16", "relu2")) == UNSUPPORTED
    assert experts(lib.make_shape(200, 128, 8, 2, 16, "bf16")) == UNSUPPORTED
    assert experts(lib.make_shape((1 << 17) + 128, 128, 8, 2, 16, "bf16")) == UNSUPPORTED
    assert experts(lib.make_shape(256, 128, 8, 2, 16, "bf16", gate_up_limit=-1.0)) == INVALID
    assert lib.load().moe_int8_experts(None, 1, A, A, A, A, A, A, A, A, A, 1 << 40, None) == INVALID
    sizes = [lib.moe_int8_experts_workspace_bytes(lib.make_shape(256, 128, 8, 2, T, "bf16")) for T in range(1, 300)]
    assert sizes == sorted(sizes) and sizes[0] > 0


NORM = ["T", "H", "k", "y", "w", "shared", "gate", "res", "post", "next", "eps", "scale", "out", "normed"]


def norm(**kw):
    a = dict(T=2, H=64, k=2, y=A, w=A, shared=A, gate=A, res=A, post=A, next=A, eps=1e-6, scale=1.0, out=A, normed=A)
    a.update(kw)
    return lib.load().moe_combine_norm(*[a[n] for n in NORM], None)


SIZES = [({"T": -1}, INVALID), ({"H": 0}, UNSUPPORTED), ({"H": 60}, UNSUPPORTED), ({"H": 16392}, UNSUPPORTED),
         ({"k": -1}, UNSUPPORTED), ({"k": 33}, UNSUPPORTED), ({"T": (1 << 23) + 1}, UNSUPPORTED),
         ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"eps": float("inf")}, INVALID),
         ({"scale": float("nan")}, INVALID), ({"scale": float("-inf")}, INVALID),
         ({"y": None}, INVALID), ({"w": None}, INVALID), ({"k": 0}, INVALID),
         ({"k": 0, "y": None, "w": None, "shared": None, "gate": None}, INVALID), ({"shared": None}, INVALID),
         ({"y": A + 8}, INVALID), ({"shared": A + 2}, INVALID), ({"post": A + 4}, INVALID), ({"next": A + 8}, INVALID),
         ({"w": A + 2}, INVALID), ({"gate": A + 1}, INVALID)]


@pytest.mark.parametrize("kw,status", SIZES + [
    ({"T": 0, "y": None, "out": None}, OK), ({"out": None}, INVALID), ({"next": None}, INVALID),
    ({"normed": None}, INVALID), ({"res": A + 8}, INVALID), ({"out": A + 8}, INVALID), ({"normed": A + 2}, INVALID),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


GRAD = ["T", "H", "k", "y", "w", "shared", "gate", "out", "post", "next", "eps", "scale", "d_out", "d_normed", "d_res",
        "d_y", "d_w", "d_shared", "d_gate", "d_post", "d_next", "ws", "nbytes"]


def norm_grad(**kw):
    a = dict(T=2, H=64, k=2, eps=1e-6, scale=1.0, nbytes=1 << 30)
    a.update({n: A for n in GRAD if n not in a})
    a.update(kw)
    return lib.load().moe_combine_norm_backward(*[a[n] for n in GRAD], None)


@pytest.mark.parametrize("kw,status", SIZES + [
    ({"T": 0, "y": None, "d_out": None}, OK), ({"out": None}, INVALID), ({"next": None}, INVALID),
    ({"d_normed": None}, INVALID), ({"d_next": None}, INVALID), ({"d_post": None}, INVALID), ({"post": None}, INVALID),
    ({"next": None, "d_next": None, "d_normed": None, "d_out": None}, INVALID),
    ({"k": 0, "y": None, "w": None}, INVALID), ({"k": 0, "y": None, "w": None, "d_y": None}, INVALID),
    ({"shared": None, "gate": None, "d_gate": None}, INVALID), ({"gate": None}, INVALID),
    ({"d_out": A + 8}, INVALID), ({"d_normed": A + 8}, INVALID), ({"d_res": A + 8}, INVALID), ({"d_y": A + 8}, INVALID),
    ({"d_shared": A + 8}, INVALID), ({"out": A + 8}, INVALID), ({"d_w": A + 2}, INVALID), ({"d_gate": A + 2}, INVALID),
    ({"d_post": A + 2}, INVALID), ({"d_next": A + 2}, INVALID), ({"ws": None}, INVALID), ({"ws": A + 128}, INVALID),
    ({"nbytes": 512}, WORKSPACE),
])
def test_norm_gradient_refusals(kw, status):
    assert norm_grad(**kw) == status


def test_norm_gradient_workspace():
    f = lib.moe_combine_norm_backward_workspace_bytes
    assert f(0, 64) == 0 and f(5, 60) == 0 and f(5, 16392) == 0 and f((1 << 24) + 1, 64) == 0
    sizes = [f(T, 64) for T in (1, 2, 100, 255, 256, 257, 511, 512, 513, 5000, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    for H in (8, 16, 504, 512, 520, 1024, 2048, 8192, 8200, 16384):  # both norms' parts of every block
        assert f(1, H) >= 8 * H and f(1 << 20, H) >= 256 * 8 * H, H


def test_tiled_products_use_no_scratch():
    """The tiled products count their loads in flight, which hold no operation that the compiler adds: none of those
    kernels may keep registers in memory."""
    import struct

    msgpack = pytest.importorskip("msgpack")
    with open(lib.LIB_PATH, "rb") as f:
        data = f.read()
    at, kernels = 0, {}
    while (at := data.find(b"AMDGPU\0", at)) >= 0:
        name, size, kind = struct.unpack("<III", data[at - 12:at])
        if name == 7 and kind == 32:  # a code object's note of its kernels
            for k in msgpack.unpackb(data[at + 8:at + 8 + size])["amdhsa.kernels"]:
                kernels[k[".name"]] = k[".private_segment_fixed_size"]
        at += 7
    tiled = {n: v for n, v in kernels.items() if "int8_tile" in n or "int8_split" in n}
    assert len(tiled) >= 12 and not any(tiled.values()), tiled
