"""Products on 8-bit integer weights against the oracle.

linear: sums are exact integers, and the three fp32 roundings behind them and the
one to bf16 are the definition's: outputs are equal bit for bit, whatever kernel the
size takes.

experts: gate and up values are equal bit for bit too; h = silu(g) u goes through an
exponential (relative error up to (|g| + 8) 2^-23 with its product, sum and
division) and is rounded to bf16.  Where no h of a row is that near to a border
between two bf16 values, its bits are the oracle's and so is y.  In the other rows
an h may be a bf16 step (2^-7 of it) away and, where it is the row's largest, move
all of the row's codes by one and its scale by 2^-7: each dequantised h is then off
by at most (1 + 2^-7) scale + 2^-7 |h|, y by the sum of those times |w| and 2^-8 of
itself."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import codecs, int8

pytestmark = pytest.mark.gpu


def _weights(rng, *shape):
    return rng.integers(-127, 128, shape).astype(np.int8), (rng.random(shape[:-1]) * 1e-3 + 1e-4).astype(np.float32)


def _x(rng, M, K):
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(1, K // 64))] *= 20
    return codecs.bf16_encode(x)


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _linear(x, c, s, stride=None, ostride=None, fill=7.0):
    d, M, K, N = gh.dev(), x.shape[0], x.shape[1], c.shape[0]
    xd = torch.full((M, stride or K), float("nan"), dtype=torch.bfloat16, device=d)
    xd[:, :K] = gh.to_device_x(x)
    out = torch.full((M + 1, ostride or N), fill, dtype=torch.bfloat16, device=d)
    ws = torch.full((lib.moe_int8_linear_workspace_bytes(M, N, K),), 0xFF, dtype=torch.uint8, device=d)
    lib.moe_int8_linear(M, N, K, torch.from_numpy(c).to(d), torch.from_numpy(s).to(d), xd, out, ws, x_stride=stride,
                        out_stride=ostride)
    torch.cuda.synchronize()
    assert (out[M] == fill).all() and (out[:M, N:] == fill).all()
    return _bits(out[:M, :N])


SIZES = [(1, 1, 16), (1, 7, 48), (2, 130, 272), (5, 64, 128), (8, 200, 2048), (1, 2816, 4096), (16, 96, 7168),
         (17, 576, 2304), (31, 50, 144), (32, 257, 1040), (33, 64, 512), (64, 320, 4096), (65, 1000, 272), (100, 513, 640),
         (129, 128, 1152), (200, 300, 4112), (256, 256, 256), (300, 2000, 2000), (511, 1408, 768), (1030, 700, 1296),
         (2100, 257, 144), (700, 4100, 2064),
         (17, 576, 7168), (70, 203, 6000), (128, 301, 4096)]  # the last three: K in runs


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(M, N, K):
    rng = np.random.default_rng(M * 7 + N)
    c, s = _weights(rng, N, K)
    x = _x(rng, M, K)
    assert np.array_equal(_linear(x, c, s), codecs.bf16_encode(int8.linear32(x, c, s)))


@pytest.mark.parametrize("M", [3, 20, 90, 400])
def test_linear_strides(M):
    rng = np.random.default_rng(M)
    c, s = _weights(rng, 301, 272)
    x = _x(rng, M, 272)
    ref = codecs.bf16_encode(int8.linear32(x, c, s))
    for stride, ostride in ((280, 304), (272, 303), (512, 301), (288, 1001)):
        assert np.array_equal(_linear(x, c, s, stride, ostride), ref)


def test_linear_of_the_batch_around_it():
    """A token's bits are the same in every batch."""
    rng = np.random.default_rng(1)
    c, s = _weights(rng, 513, 2064)
    x = _x(rng, 600, 2064)
    full = _linear(x, c, s)
    for M in (1, 4, 16, 17, 32, 33, 63, 64, 65, 130, 257):
        assert np.array_equal(_linear(x[:M], c, s), full[:M]), M


@pytest.mark.parametrize("M", [1, 20, 80])
def test_linear_largest_sums(M):
    """Codes of -128 and 127 over the longest K: sums of 128 127 2^17 = 0.99 2^31."""
    K = 1 << 17
    c = np.full((5, K), -128, np.int8)
    c[1], c[2, ::2] = 127, 127
    s = np.ones(5, np.float32)
    x = codecs.bf16_encode(np.ones((M, K), np.float32))
    x[M // 2] |= 0x8000
    ref = codecs.bf16_encode(int8.linear32(x, c, s))
    assert np.array_equal(_linear(x, c, s), ref)


@pytest.mark.parametrize("M", [4, 24, 70, 300, 1100])
def test_linear_of_odd_rows(M):
    """Zero rows, rows of tiny and of the largest values; rows that are not finite give NaN, and nothing elsewhere."""
    rng = np.random.default_rng(M)
    c, s = _weights(rng, 140, 400)
    x = _x(rng, M, 400)
    x[1::9] = 0
    x[2::9] = codecs.bf16_encode((rng.standard_normal((len(x[2::9]), 400)) * 1e-34).astype(np.float32))
    x[3::9, 5] = 0x7F7F
    ref = codecs.bf16_encode(int8.linear32(x, c, s))
    bad = np.arange(M) % 10 == 0
    x[0::20, 399], x[10::20, 7] = 0x7F80, 0xFFC1
    got = _linear(x, c, s)
    assert np.array_equal(got[~bad], ref[~bad])
    assert np.isnan(codecs.bf16_decode(got[bad])).all()


def test_quantize_weights():
    rng = np.random.default_rng(2)
    d = gh.dev()
    for count, rows, K in ((1, 1, 16), (3, 5, 272), (2, 130, 4112)):
        w = (rng.standard_normal((count, rows, K)) * 0.02).astype(np.float32)
        w[0, 0] = 0
        c = torch.full((count, rows, K), 99, dtype=torch.int8, device=d)
        s = torch.full((count, rows), 99.0, device=d)
        lib.moe_int8_quantize_weights(count, rows, K, torch.from_numpy(w).to(d), c, s)
        rc, rs = int8.quantize_rows(w.reshape(-1, K))
        assert np.array_equal(c.cpu().numpy().reshape(-1, K), rc) and np.array_equal(s.cpu().numpy().reshape(-1), rs)
    w[0, 3, 9], w[1, 7, 0] = np.nan, -np.inf
    lib.moe_int8_quantize_weights(2, 130, 4112, torch.from_numpy(w).to(d), c, s)
    bad = torch.isnan(s).cpu().numpy()
    assert bad.sum() == 2 and bad[0, 3] and bad[1, 7]
    assert np.array_equal(c.cpu().numpy().reshape(-1, K)[~bad.reshape(-1)], rc[~bad.reshape(-1)])


# ------------------------------------------------------------------ experts


def _routing(rng, T, E, k, skew):
    z = rng.standard_normal((T, E)) + skew * rng.standard_normal(E)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    flat = ids.reshape(-1)
    return np.r_[0, np.cumsum(np.bincount(flat, minlength=E))].astype(np.int32), np.argsort(flat, kind="stable").astype(np.int32)


def _experts(x, w13, s13, w2, s2, off, pairs, k, limit=0.0, max_tokens=None):
    d, T, H, E, I = gh.dev(), x.shape[0], x.shape[1], w13.shape[0], w2.shape[2]
    shape = lib.make_shape(H, I, E, k, max_tokens or T, "bf16", gate_up_limit=limit)
    ws = torch.full((lib.moe_int8_experts_workspace_bytes(shape),), 0xFF, dtype=torch.uint8, device=d)
    y = torch.full((T * k + 1, H), 7.0, dtype=torch.bfloat16, device=d)
    lib.moe_int8_experts(shape, T, *(torch.from_numpy(v).to(d) for v in (w13, s13, w2, s2, off, pairs)),
                         gh.to_device_x(x), y, ws)
    torch.cuda.synchronize()
    assert (y[T * k] == 7.0).all()
    return _bits(y[:T * k])


def _near(gate, hid):
    """Whether an h is within its error of a border between two bf16 values, [P, I]."""
    h = np.abs(hid)
    with np.errstate(divide="ignore"):
        step = 2.0 ** (np.floor(np.log2(np.where(h > 0, h, 1.0))) - 7)
    pos = h / step
    return np.abs(pos - np.floor(pos) - 0.5) * step <= h * (np.abs(gate) + 8) * 2.0 ** -23


def _check_experts(got, ref, w2, s2, off, pairs):
    y, gate, _, hid = ref
    near = _near(gate, hid).any(axis=1)  # by sorted row
    bits = codecs.bf16_encode(y)
    same = (got == bits).all(axis=1)
    assert same[pairs[~near]].all(), "a row whose intermediate is certain differs"
    g, r = codecs.bf16_decode(got).astype(np.float64), y.astype(np.float64)
    for e in range(w2.shape[0]):
        rows = np.arange(off[e], off[e + 1])
        rows = rows[near[rows]]
        if len(rows):
            h = np.abs(hid[rows])
            scale = np.maximum(h.max(axis=1, keepdims=True), 2.0 ** -100) / 127 * (1 + 2.0 ** -7)
            tol = ((1 + 2.0 ** -7) * scale + 2.0 ** -7 * h) @ (np.abs(w2[e].astype(np.float64)) * s2[e][:, None]).T
            p = pairs[rows]
            assert (np.abs(g[p] - r[p]) <= tol + 2.0 ** -8 * np.abs(r[p])).all()
    return near.mean()


CASES = [  # T, H, I, E, k, skew, limit: the streaming kernel's sources, the tiles of 64, 128 and 256 rows
    (1, 256, 128, 8, 2, 0.0, 0.0), (1, 1024, 256, 16, 8, 0.0, 2.0), (3, 384, 128, 5, 3, 1.0, 0.0),
    (8, 2048, 256, 12, 6, 0.0, 0.0), (9, 512, 128, 64, 8, 3.0, 0.0), (40, 4096, 128, 4, 2, 0.0, 1.0),
    (30, 256, 128, 2, 1, 0.0, 0.0), (64, 512, 768, 60, 4, 1.0, 0.0), (333, 512, 384, 16, 3, 0.5, 0.0),
    (500, 256, 256, 7, 2, 2.0, 3.0), (700, 384, 512, 6, 2, 1.0, 0.0), (1, 16640, 128, 4, 2, 0.0, 0.0),
    (6, 256, 16640, 4, 2, 0.0, 0.0), (120, 512, 768, 40, 4, 0.5, 0.0), (90, 256, 256, 6, 2, 1.0, 0.0),
    (14, 4096, 128, 2, 1, 0.0, 0.0), (250, 384, 1408, 24, 4, 0.5, 1.0),
]


@pytest.mark.parametrize("T,H,I,E,k,skew,limit", CASES)
def test_experts(T, H, I, E, k, skew, limit):
    rng = np.random.default_rng(T * 3 + E)
    (w13, s13), (w2, s2) = _weights(rng, E, 2 * I, H), _weights(rng, E, H, I)
    s13 = (s13 * np.float32(30.0 / np.sqrt(H))).astype(np.float32)
    off, pairs = _routing(rng, T, E, k, skew)
    x = _x(rng, T, H)
    got = _experts(x, w13, s13, w2, s2, off, pairs, k, limit)
    _check_experts(got, int8.experts(x, w13, s13, w2, s2, off, pairs, k, limit), w2, s2, off, pairs)
    assert np.array_equal(_experts(x, w13, s13, w2, s2, off, pairs, k, limit, max_tokens=T + 100), got)


def test_experts_of_the_batch_around_them():
    """A token's rows are the same bits alone and in a batch of any size."""
    rng = np.random.default_rng(8)
    H, I, E, k, T = 512, 256, 8, 2, 600
    (w13, s13), (w2, s2) = _weights(rng, E, 2 * I, H), _weights(rng, E, H, I)
    x = _x(rng, T, H)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]

    def run(n):
        flat = ids[:n].reshape(-1)
        off = np.r_[0, np.cumsum(np.bincount(flat, minlength=E))].astype(np.int32)
        return _experts(x[:n], w13, s13, w2, s2, off, np.argsort(flat, kind="stable").astype(np.int32), k)

    full = run(T)
    for n in (1, 3, 8, 20, 100, 260):
        assert np.array_equal(run(n), full[:n * k]), n


@pytest.mark.parametrize("T", [2, 40, 300])
def test_experts_rows_that_are_not_finite(T):
    rng = np.random.default_rng(T)
    H, I, E, k = 256, 128, 6, 2
    (w13, s13), (w2, s2) = _weights(rng, E, 2 * I, H), _weights(rng, E, H, I)
    off, pairs = _routing(rng, T, E, k, 0.0)
    x = _x(rng, T, H)
    for limit in (0.0, 1.0):
        good = _experts(x, w13, s13, w2, s2, off, pairs, k, limit)
        z = x.copy()
        z[0, 9], z[T // 2, 200] = 0x7FC0, 0xFF80
        got = _experts(z, w13, s13, w2, s2, off, pairs, k, limit)
        bad = np.zeros(T, bool)
        bad[[0, T // 2]] = True
        bad = np.repeat(bad, k)
        assert np.array_equal(got[~bad], good[~bad]) and np.isnan(codecs.bf16_decode(got[bad])).all()


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(9)
    d, H, I, E, k = gh.dev(), 1024, 256, 16, 4
    (w13, s13), (w2, s2) = _weights(rng, E, 2 * I, H), _weights(rng, E, H, I)
    dw = [torch.from_numpy(v).to(d) for v in (w13, s13, w2, s2)]
    for T in (2, 50, 400):
        off, pairs = (torch.from_numpy(v).to(d) for v in _routing(rng, T, E, k, 0.5))
        shape = lib.make_shape(H, I, E, k, T, "bf16")
        x = gh.to_device_x(_x(rng, T, H))
        xs = [x, x.flip(0).contiguous(), (x * 2).contiguous()]
        ws = [torch.empty(lib.moe_int8_experts_workspace_bytes(shape), dtype=torch.uint8, device=d) for _ in range(2)]
        lw = [torch.empty(lib.moe_int8_linear_workspace_bytes(T * k, 2 * I, H), dtype=torch.uint8, device=d) for _ in range(2)]
        outs = [(torch.zeros(T * k, H, dtype=torch.bfloat16, device=d), torch.zeros(T * k, 2 * I, dtype=torch.bfloat16, device=d))
                for _ in range(2)]

        def step(i, inp):
            lib.moe_int8_experts(shape, T, *dw, off, pairs, inp, outs[i][0], ws[i])
            lib.moe_int8_linear(T * k, 2 * I, H, dw[0], dw[1], outs[i][0], outs[i][1], lw[i])

        step(0, x)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(1, x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        hold = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(1, hold)
        for inp in xs:
            hold.copy_(inp)
            ws[1].fill_(0xFF)
            lw[1].fill_(0xFF)
            graph.replay()
            step(0, inp)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_rows_far_apart():
    """x and out rows past 2^31 values: 70000 rows 32768 apart."""
    rng = np.random.default_rng(10)
    d, M, K, N, ld = gh.dev(), 70000, 144, 40, 32768
    c, s = _weights(rng, N, K)
    x = torch.empty(M, ld, dtype=torch.bfloat16, device=d)
    x[:, :K].normal_(generator=torch.Generator(device=d).manual_seed(3))
    out = torch.empty(M, ld, dtype=torch.bfloat16, device=d)
    ws = torch.empty(lib.moe_int8_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device=d)
    lib.moe_int8_linear(M, N, K, torch.from_numpy(c).to(d), torch.from_numpy(s).to(d), x, out, ws, x_stride=ld, out_stride=ld)
    torch.cuda.synchronize()
    for at in (slice(0, 70), slice(65500, 65600), slice(M - 70, M)):
        ref = codecs.bf16_encode(int8.linear32(_bits(x[at, :K]), c, s))
        assert np.array_equal(_bits(out[at, :N]), ref)


@pytest.mark.parametrize("T", [2, 60, 1100])
def test_experts_weights_past_2_31(T):
    """260 experts of 2^23 + 2^22 codes: 3 2^30 of them; the last ones' rows."""
    d, H, I, E, k = gh.dev(), 4096, 1024, 260, 2
    g = torch.Generator(device=d).manual_seed(4)
    w13 = torch.randint(-127, 128, (E, 2 * I, H), generator=g, device=d, dtype=torch.int8)
    w2 = torch.randint(-127, 128, (E, H, I), generator=g, device=d, dtype=torch.int8)
    rng = np.random.default_rng(11)
    s13 = (rng.random((E, 2 * I)) * 1e-3).astype(np.float32)
    s2 = (rng.random((E, H)) * 1e-3).astype(np.float32)
    x = _x(rng, T, H)
    used = np.array([0, 128, 255, 258, 259])
    flat = used[rng.integers(0, 5, T * k)]
    off = np.r_[0, np.cumsum(np.bincount(flat, minlength=E))].astype(np.int32)
    pairs = np.argsort(flat, kind="stable").astype(np.int32)
    shape = lib.make_shape(H, I, E, k, T, "bf16")
    ws = torch.empty(lib.moe_int8_experts_workspace_bytes(shape), dtype=torch.uint8, device=d)
    y = torch.empty(T * k, H, dtype=torch.bfloat16, device=d)
    lib.moe_int8_experts(shape, T, w13, torch.from_numpy(s13).to(d), w2, torch.from_numpy(s2).to(d),
                         torch.from_numpy(off).to(d), torch.from_numpy(pairs).to(d), gh.to_device_x(x), y, ws)
    small = np.searchsorted(used, flat)
    off5 = np.r_[0, np.cumsum(np.bincount(small, minlength=5))].astype(np.int32)
    pick = torch.from_numpy(used).to(d)
    a13, a2 = w13[pick].cpu().numpy(), w2[pick].cpu().numpy()
    _check_experts(_bits(y), int8.experts(x, a13, s13[used], a2, s2[used], off5, pairs, k), a2, s2[used], off5, pairs)


def test_experts_of_more_than_2_31_values():
    """16400 tokens of 131072 values: a token's rows are the same bits as in a batch of 300 (whose rows other kernels read
    by 32-bit offsets)."""
    d, H, I, E, k, T, n = gh.dev(), 1 << 17, 128, 3, 1, 16400, 300
    g = torch.Generator(device=d).manual_seed(6)
    w13 = torch.randint(-127, 128, (E, 2 * I, H), generator=g, device=d, dtype=torch.int8)
    w2 = torch.randint(-127, 128, (E, H, I), generator=g, device=d, dtype=torch.int8)
    s13 = torch.rand(E, 2 * I, generator=g, device=d) * 1e-5
    s2 = torch.rand(E, H, generator=g, device=d) * 1e-3
    x = torch.empty(T, H, dtype=torch.bfloat16, device=d).normal_(generator=g)
    flat = torch.randint(0, E, (T,), generator=g, device=d)

    def run(x, flat):
        T = len(flat)
        shape = lib.make_shape(H, I, E, k, T, "bf16")
        off = torch.zeros(E + 1, dtype=torch.int32, device=d)
        off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
        ws = torch.empty(lib.moe_int8_experts_workspace_bytes(shape), dtype=torch.uint8, device=d)
        y = torch.full((T, H), 7.0, dtype=torch.bfloat16, device=d)
        lib.moe_int8_experts(shape, T, w13, s13, w2, s2, off, flat.argsort(stable=True).int(), x, y, ws)
        return y

    y = run(x, flat)
    for at in (slice(0, n), slice(T - n, T)):
        assert torch.equal(y[at].view(torch.int16), run(x[at].contiguous(), flat[at]).view(torch.int16))
        assert (y[at] != 7.0).any(dim=1).all()
