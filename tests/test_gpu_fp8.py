"""Products on block-128 fp8 weights against the float64 oracle.

Tolerances.  linear: the bf16 output is off by half a step, 2^-8 |y|.  The fp8
matrix instruction adds products in groups of 8 consecutive K, each product cut
to 13 bits below the exponent of the group's largest (measured: beside 2^16 a
product of 14.06 counts as 8, one below 8 as 0, of either sign; products of
other groups are not touched), so a group's sum is off by less than 7 * 2^-13
of its largest product; fp32 sums of fewer than 2^8 such parts add 2^-16 of
their sizes at most, together 2^-10 of the groups' largest products.  That is a
bound of the worst case; cut parts have random signs, so over all values the
error has to stay in the root mean square within 2^-8 / sqrt 3 of the outputs
(a value's rounding error is at most 2^-8 of it and evenly spread) and 2^-14 of
the same sum.  experts: the same output rounding (rms 2^-8 / sqrt 3 = 2.3e-3)
and, where the gate and up sums' error (2^-16 each) carries the intermediate
over a border between two codes (borders are at least 2^-4 apart, a code steps
by at most 2^-3 of the value): a share of at most 2 * 2^-15 / 2^-4 = 2^-10 of
the values steps, in the root mean square 2^-5 * 2^-3 = 3.9e-3 of the sum;
together 4.6e-3, held to 6e-3."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import codecs, fp8_block as fb, moe

pytestmark = pytest.mark.gpu

BITS = 2.0 ** -8


def _weights(rng, N, K):
    return fb.quantize_weights((rng.standard_normal((N, K)) * 0.02).astype(np.float32))


def _x(rng, M, K):
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(1, K // 64))] *= 20
    return codecs.bf16_encode(x)


def _linear(x, c, s, stride=None, ostride=None, fill=7.0):
    """(out float64, the whole out buffer) through the library."""
    d, M, K, N = gh.dev(), x.shape[0], x.shape[1], c.shape[0]
    xd = torch.full((M, stride or K), float("nan"), dtype=torch.bfloat16, device=d)
    xd[:, :K] = gh.to_device_x(x)
    out = torch.full((M + 1, ostride or N), fill, dtype=torch.bfloat16, device=d)
    ws = torch.full((lib.moe_fp8_linear_workspace_bytes(M, N, K),), 0xFF, dtype=torch.uint8, device=d)
    lib.moe_fp8_linear(M, N, K, torch.from_numpy(c).to(d), torch.from_numpy(s).to(d), xd, out, ws, x_stride=stride,
                       out_stride=ostride)
    torch.cuda.synchronize()
    return out[:M, :N].double().cpu().numpy(), out


def _check(got, ref, groups):
    bad = np.abs(got - ref) > BITS * np.abs(ref) + 2.0 ** -10 * groups
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    assert np.linalg.norm(got - ref) <= BITS / np.sqrt(3) * np.linalg.norm(ref) + 2.0 ** -14 * np.linalg.norm(groups)


@pytest.mark.parametrize("count,rows,K", [(1, 1, 16), (2, 130, 144), (3, 128, 256), (1, 257, 400)])
def test_quantize_weights_is_the_oracles(count, rows, K):
    rng = np.random.default_rng(rows + K)
    w = (rng.standard_normal((count, rows, K)) * 0.02).astype(np.float32)
    w[0, 0, :16] = 0
    d = gh.dev()
    codes = torch.empty(count, rows, K, dtype=torch.uint8, device=d)
    scales = torch.empty(count, -(-rows // 128), -(-K // 128), device=d)
    lib.moe_fp8_quantize_weights(count, rows, K, torch.from_numpy(w).to(d), codes, scales)
    for i in range(count):
        c, s = fb.quantize_weights(w[i])
        assert np.array_equal(codes[i].cpu().numpy() & 0x7F, c & 0x7F), i  # a rounded zero keeps its sign on the GPU
        assert np.array_equal(codecs.e4m3_decode(codes[i].cpu().numpy()), codecs.e4m3_decode(c))
        assert np.array_equal(scales[i].cpu().numpy(), s)


SIZES = [(1, 1, 16), (1, 5, 2048), (2, 64, 128), (3, 130, 144), (16, 129, 400), (17, 576, 1040), (31, 67, 272),
         (33, 256, 256), (64, 200, 1024), (100, 128, 128), (128, 384, 640), (129, 257, 272), (255, 300, 512),
         (256, 256, 1024), (257, 512, 384), (300, 520, 2064), (513, 1030, 144),
         # long K over many waves; more tiles than compute units for each tile shape in turn
         (9, 100, 4112), (16, 130, 2048), (32, 70, 4096), (300, 2000, 272), (700, 2000, 400), (1000, 2900, 144),
         (2100, 4100, 272)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(M, N, K):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    x, (c, s) = _x(rng, M, K), _weights(rng, N, K)
    got, out = _linear(x, c, s)
    _check(got, *fb.linear(x, c, s))
    assert bool((out[M] == 7.0).all())  # the row behind the last one is left alone


# K split over blocks as well (few weight rows, a long K; the last run shorter), with its neighbours that are not split:
# one row, more weight rows, a K of fewer than 16 blocks, more token rows
RUNS = [(2, 16, 8208), (5, 7, 5136), (16, 100, 16400), (17, 577, 7168), (40, 33, 2064), (64, 1000, 1040), (128, 250, 4112),
        (128, 16, 32768), (1, 40, 8208), (20, 4100, 1040), (12, 4100, 4112), (64, 100, 912), (129, 250, 4112)]


@pytest.mark.parametrize("M,N,K", RUNS)
def test_linear_runs_of_k(M, N, K):
    rng = np.random.default_rng(M * 131 + N + K)
    x, (c, s) = _x(rng, M, K), _weights(rng, N, K)
    got, out = _linear(x, c, s, K + 8, N + 3)
    _check(got, *fb.linear(x, c, s))
    assert bool((out[:, N:] == 7.0).all()) and bool((out[M] == 7.0).all())


def test_linear_one_workspace_for_fewer_rows():
    """The bytes for max_M rows serve every smaller number, of whichever kernels."""
    rng, N, K, d = np.random.default_rng(8), 144, 4112, gh.dev()
    x, (c, s) = _x(rng, 140, K), _weights(rng, N, K)
    cd, sd, xd = torch.from_numpy(c).to(d), torch.from_numpy(s).to(d), gh.to_device_x(x)
    ref, groups = fb.linear(x, c, s)
    size = [lib.moe_fp8_linear_workspace_bytes(m, N, K) for m in range(1, 141)]
    assert size == sorted(size)
    ws = torch.full((size[-1],), 0xFF, dtype=torch.uint8, device=d)
    for M in (140, 1, 128, 3, 16, 33):
        out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=d)
        lib.moe_fp8_linear(M, N, K, cd, sd, xd, out, ws)
        torch.cuda.synchronize()
        _check(out[:M].double().cpu().numpy(), ref[:M], groups[:M])
        assert bool((out[M] == 7.0).all())


@pytest.mark.parametrize("M,N,K", [(1, 130, 144), (20, 96, 256), (300, 130, 400), (512, 512, 512)])
@pytest.mark.parametrize("odd", [1, 8])
def test_linear_strides(M, N, K, odd):
    """Wider rows on both sides (an out stride that breaks 4- and 16-byte alignment too); the columns between stay."""
    rng = np.random.default_rng(M + N)
    x, (c, s) = _x(rng, M, K), _weights(rng, N, K)
    got, out = _linear(x, c, s, K + 24, N + odd)
    _check(got, *fb.linear(x, c, s))
    assert bool((out[:, N:] == 7.0).all()) and bool((out[M] == 7.0).all())


@pytest.mark.parametrize("M", [3, 300])
def test_linear_out_not_aligned(M):
    rng = np.random.default_rng(5)
    N, K, d = 264, 256, gh.dev()
    x, (c, s) = _x(rng, M, K), _weights(rng, N, K)
    flat = torch.full((M * N + 8,), 7.0, dtype=torch.bfloat16, device=d)
    out = flat[1:1 + M * N].view(M, N)
    ws = torch.empty(lib.moe_fp8_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device=d)
    lib.moe_fp8_linear(M, N, K, torch.from_numpy(c).to(d), torch.from_numpy(s).to(d), gh.to_device_x(x), out, ws)
    _check(out.double().cpu().numpy(), *fb.linear(x, c, s))
    assert flat[0].item() == 7.0 and bool((flat[1 + M * N:] == 7.0).all())


@pytest.mark.parametrize("M", [4, 300])
def test_linear_special_values(M):
    """Zero rows, tiny rows, wide ranges inside a block, infinities and NaN; NaN weight codes behind K."""
    rng = np.random.default_rng(6)
    N, K = 256, 400
    x, (c, s) = _x(rng, M, K), _weights(rng, N, K)
    xf = codecs.bf16_decode(x).copy()
    xf[0] = 0.0
    xf[1] = xf[1] * 2.0 ** -110  # below the smallest magnitude that sets a scale
    xf[2, 130] = 3e38
    x = codecs.bf16_encode(xf.astype(np.float32))
    got, _ = _linear(x, c, s)
    ref, groups = fb.linear(x, c, s)
    assert not got[0].any()
    with np.errstate(over="ignore"):
        _check(got, ref, groups)
    for bad in (np.inf, -np.inf, np.nan):
        xt = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).clone()
        xt[3, 399] = bad
        got, _ = _linear(xt.view(torch.int16).numpy().view(np.uint16), c, s)
        assert np.isnan(got[3]).all()
        keep = np.arange(M) != 3
        _check(got[keep], ref[keep], groups[keep])
    c2 = c.copy()
    c2[7, 399] = 0x7F  # a NaN code makes its own column NaN, not its neighbours'
    got, _ = _linear(x, c2, s)
    assert np.isnan(got[:, 7]).all()
    keep = np.arange(N) != 7
    _check(got[:, keep], ref[:, keep], groups[:, keep])


@pytest.mark.parametrize("M", [4, 20])
def test_linear_runs_of_k_special_values_and_captured(M):
    """K split over blocks: infinities and NaN in any run spoil their own row only; replays give the eager bits."""
    rng, d = np.random.default_rng(16), gh.dev()
    N, K = 100, 4112
    x, (c, s) = _x(rng, M, K), _weights(rng, N, K)
    xf = codecs.bf16_decode(x).copy()
    xf[0] = 0.0
    x = codecs.bf16_encode(xf.astype(np.float32))
    ref, groups = fb.linear(x, c, s)
    keep = np.arange(M) != 3
    for bad, col in ((np.inf, 0), (-np.inf, 2047), (np.nan, 4111)):
        xt = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).clone()
        xt[3, col] = bad
        got, _ = _linear(xt.view(torch.int16).numpy().view(np.uint16), c, s)
        assert np.isnan(got[3]).all() and not got[0].any()
        _check(got[keep], ref[keep], groups[keep])
    cd, sd, xd = torch.from_numpy(c).to(d), torch.from_numpy(s).to(d), gh.to_device_x(x)
    ws = torch.empty(lib.moe_fp8_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device=d)
    out, eager = (torch.empty(M, N, dtype=torch.bfloat16, device=d) for _ in range(2))
    lib.moe_fp8_linear(M, N, K, cd, sd, xd, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.moe_fp8_linear(M, N, K, cd, sd, xd, out, ws)
    for i in range(4):
        xd.mul_(-1.0 if i % 2 else 0.5)
        out.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        lib.moe_fp8_linear(M, N, K, cd, sd, xd, eager, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


@pytest.mark.parametrize("M", [2, 20, 70])
def test_linear_offsets_beyond_32_bits(M):
    """A weight matrix of over 2^31 codes, and rows of x and out over 2^32 elements apart in all: the first and the last
    columns against a float64 product on the same codes."""
    d, N, K = gh.dev(), 300032, 7168
    g = torch.Generator(device=d)
    g.manual_seed(M)
    codes = torch.empty(N, K, dtype=torch.uint8, device=d)
    for i in range(0, N, 50000):
        codes[i:i + 50000] = torch.randint(0, 0x7F, codes[i:i + 50000].shape, generator=g, device=d, dtype=torch.uint8)
    scales = 1e-4 * (0.5 + torch.rand(N // 128, K // 128, generator=g, device=d))
    x = torch.randn(M, K, generator=g, device=d).to(torch.bfloat16)
    xw = torch.empty(M, 1 << 26, dtype=torch.bfloat16, device=d)[:, :K]
    xw.copy_(x)
    out = torch.empty(M, 1 << 26, dtype=torch.bfloat16, device=d)[:, :N]
    ws = torch.empty(lib.moe_fp8_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device=d)
    lib.moe_fp8_linear(M, N, K, codes, scales, xw, out, ws, x_stride=1 << 26, out_stride=1 << 26)
    torch.cuda.synchronize()
    xh = torch.from_numpy(fb.dequantize_rows(*fb.quantize_rows(codecs.bf16_decode(gh.bf16_numpy(x))))).to(d)
    for n in (0, N // 256 * 128, N - 128):
        w = codes[n:n + 128].view(torch.float8_e4m3fn).double() * scales[n // 128].double().repeat_interleave(128)
        groups = xh.abs().view(M, -1, 8).amax(2) @ w.abs().view(128, -1, 8).amax(2).t()
        _check(out[:, n:n + 128].double().cpu().numpy(), (xh @ w.t()).cpu().numpy(), groups.cpu().numpy())


def test_linear_is_reproducible_and_captured():
    rng = np.random.default_rng(8)
    d = gh.dev()
    for M, N, K in ((1, 640, 1024), (40, 640, 1024), (400, 640, 1024)):
        c, s = (torch.from_numpy(v).to(d) for v in _weights(rng, N, K))
        xs = [gh.to_device_x(_x(rng, M, K)) for _ in range(3)]
        x = xs[0].clone()
        ws = torch.empty(lib.moe_fp8_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device=d)
        out = torch.empty(M, N, dtype=torch.bfloat16, device=d)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lib.moe_fp8_linear(M, N, K, c, s, x, out, ws)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.moe_fp8_linear(M, N, K, c, s, x, out, ws)
        for i in range(4):
            x.copy_(xs[i % 3])
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            eager = torch.empty_like(out)
            lib.moe_fp8_linear(M, N, K, c, s, x, eager, ws)
            torch.cuda.synchronize()
            assert torch.equal(out, eager), (M, i)


def test_linear_input_gradient_on_transposed_weights():
    """dx = dy . W through the same call on the transposed codes and scales, and against differences of the
    linear form sum(dy * (x . W^T)) in x."""
    rng = np.random.default_rng(9)
    M, N, K = 37, 256, 384
    c, s = _weights(rng, N, K)
    dy = _x(rng, M, N)
    ct, st = np.ascontiguousarray(c.T), np.ascontiguousarray(s.T)
    got, _ = _linear(dy, ct, st)
    ref, groups = fb.linear(dy, ct, st)
    _check(got, ref, groups)
    w = fb.dequantize_weights(c, s)
    dyh = fb.dequantize_rows(*fb.quantize_rows(codecs.bf16_decode(dy)))
    x = rng.standard_normal((M, K))
    for k in (0, 129, 383):
        h = np.zeros((M, K))
        h[:, k] = 1.0
        diff = ((dyh * ((x + h) @ w.T)).sum(1) - (dyh * ((x - h) @ w.T)).sum(1)) / 2
        assert np.all(np.abs(got[:, k] - diff) <= BITS * np.abs(diff) + 2.0 ** -10 * groups[:, k] + 1e-9)


# ------------------------------------------------------------------ experts


def _route(rng, T, E, k, only=None):
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if only is not None:
        logits[:, only] += 50.0
    return logits


def _layer(rng, H, I, E):
    q13 = [_weights(rng, 2 * I, H) for _ in range(E)]
    q2 = [_weights(rng, H, I) for _ in range(E)]
    return (np.stack([c for c, _ in q13]), np.stack([s for _, s in q13]), np.stack([c for c, _ in q2]),
            np.stack([s for _, s in q2]))


EXPERTS = [  # T, H, I, E, k, experts that take every token, gate/up clamp
    (1, 256, 128, 1, 1, None, 0.0), (1, 512, 256, 8, 8, None, 0.0), (3, 256, 128, 4, 2, [1], 0.0),
    (16, 384, 256, 8, 2, None, 0.0), (17, 256, 384, 3, 1, [2], 0.0), (33, 256, 128, 16, 4, [0, 5], 0.05),
    (64, 512, 128, 4, 2, None, 0.0), (130, 256, 256, 2, 1, None, 0.0), (300, 256, 128, 6, 2, [3], 0.1),
    (260, 384, 384, 2, 2, None, 0.0), (700, 256, 256, 4, 2, [1], 0.0), (513, 256, 128, 1, 1, None, 0.0),
    (40, 256, 128, 300, 3, None, 0.0), (24, 256, 128, 1024, 32, None, 0.0),
]


@pytest.mark.parametrize("T,H,I,E,k,only,limit", EXPERTS)
def test_experts_in_the_layer(T, H, I, E, k, only, limit):
    """route, permute, experts and combine together, each step against the oracle's on the same inputs."""
    rng = np.random.default_rng(T * 131 + E)
    d = gh.dev()
    x, logits = _x(rng, T, H), _route(rng, T, E, k, only)
    w = _layer(rng, H, I, min(E, 16))
    pick = np.arange(E) % w[0].shape[0]
    w = [v[pick] for v in w]
    shape = lib.make_shape(H, I, E, k, T + 3, "bf16", gate_up_limit=limit)
    ids = torch.empty(T, k, dtype=torch.int32, device=d)
    wts = torch.empty(T, k, device=d)
    off = torch.empty(E + 1, dtype=torch.int32, device=d)
    pairs = torch.empty(T * k, dtype=torch.int32, device=d)
    pos = torch.empty(T * k, dtype=torch.int32, device=d)
    xd = gh.to_device_x(x)
    lib.moe_route(shape, T, torch.from_numpy(logits).to(d), ids, wts)
    lib.moe_permute(shape, T, ids, xd, off, pairs, pos, xd)
    y = torch.full((T * k + 1, H), 7.0, dtype=torch.bfloat16, device=d)
    ws = torch.full((lib.moe_fp8_experts_workspace_bytes(shape),), 0xFF, dtype=torch.uint8, device=d)
    wd = [torch.from_numpy(v).to(d) for v in w]
    lib.moe_fp8_experts(shape, T, wd[0], wd[1], wd[2], wd[3], off, pairs, xd, y, ws)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=d)
    lib.moe_combine(shape, T, y, wts, out)
    torch.cuda.synchronize()
    oid, ow = moe.route(logits, k)
    assert np.array_equal(ids.cpu().numpy(), oid)
    ref = fb.experts(x, oid, *w, limit)
    got = y[:T * k].double().cpu().numpy()
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    rms = np.sqrt((ref * ref).mean())
    print(f"  T={T} H={H} I={I} E={E} k={k}: relL2 {rel:.2e} max|d|/rms {np.abs(got - ref).max() / rms:.2e}", flush=True)
    assert rel <= 6e-3 and np.abs(got - ref).max() <= 5e-2 * max(rms, np.abs(ref).max())
    assert bool((y[T * k] == 7.0).all())
    combined = (ow[:, :, None] * got.reshape(T, k, H)).sum(1)
    # one rounding to bf16, and fp32 sums of at most 32 terms
    size = (np.abs(ow)[:, :, None] * np.abs(got.reshape(T, k, H))).sum(1)
    assert np.all(np.abs(out.double().cpu().numpy() - combined) <= BITS * np.abs(combined) + 2.0 ** -18 * size)
    y2 = torch.empty_like(y)
    lib.moe_fp8_experts(shape, T, wd[0], wd[1], wd[2], wd[3], off, pairs, xd, y2, ws)
    torch.cuda.synchronize()
    assert torch.equal(y2[:T * k], y[:T * k])


@pytest.mark.parametrize("T,H,I,E,k,only,limit", [
    (1, 1024, 384, 8, 8, None, 0.0), (8, 1024, 512, 64, 6, None, 0.0), (7, 7168, 128, 4, 3, None, 0.0),
    (2, 1152, 1152, 30, 7, None, 0.0), (5, 2176, 256, 1024, 32, None, 0.0), (8, 512, 4096, 6, 2, [2], 0.05),
    # rows whose codes do not fit LDS: quantised by every wave, tiles of 16 and of 32 rows
    (8, 8192, 128, 4, 2, None, 0.0), (40, 8192, 128, 2, 1, [0], 0.0),
])
def test_experts_of_few_tokens(T, H, I, E, k, only, limit):
    test_experts_in_the_layer(T, H, I, E, k, only, limit)


@pytest.mark.parametrize("T", [3, 8, 100])
def test_experts_picked_twice_by_a_token(T):
    """An expert may hold more rows than there are tokens."""
    rng = np.random.default_rng(T)
    d, (H, I, E, k) = gh.dev(), (384, 256, 5, 4)
    x, w = _x(rng, T, H), _layer(rng, H, I, E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[::2] = 3
    shape = lib.make_shape(H, I, E, k, T, "bf16")
    off = torch.empty(E + 1, dtype=torch.int32, device=d)
    pairs, pos = (torch.empty(T * k, dtype=torch.int32, device=d) for _ in range(2))
    xd = gh.to_device_x(x)
    lib.moe_permute(shape, T, torch.from_numpy(ids).to(d), xd, off, pairs, pos, xd)
    y = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device=d)
    ws = torch.full((lib.moe_fp8_experts_workspace_bytes(shape),), 0xFF, dtype=torch.uint8, device=d)
    lib.moe_fp8_experts(shape, T, *(torch.from_numpy(v).to(d) for v in w), off, pairs, xd, y, ws)
    torch.cuda.synchronize()
    ref = fb.experts(x, ids, *w, 0.0)
    got = y.double().cpu().numpy()
    assert np.linalg.norm(got - ref) <= 6e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("T", [3, 40, 400])
def test_experts_of_a_token_that_is_not_finite(T):
    """NaN in every row of that token, nothing in the others (which share experts, tiles and blocks with it)."""
    rng = np.random.default_rng(T)
    d, (H, I, E, k) = gh.dev(), (512, 256, 4, 2)
    w = [torch.from_numpy(v).to(d) for v in _layer(rng, H, I, E)]
    ids = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).to(d)
    shape = lib.make_shape(H, I, E, k, T, "bf16")
    off = torch.empty(E + 1, dtype=torch.int32, device=d)
    pairs, pos = (torch.empty(T * k, dtype=torch.int32, device=d) for _ in range(2))
    ws = torch.full((lib.moe_fp8_experts_workspace_bytes(shape),), 0xFF, dtype=torch.uint8, device=d)
    x = gh.to_device_x(_x(rng, T, H))
    lib.moe_permute(shape, T, ids, x, off, pairs, pos, x)
    ys = []
    for bad in (0.0, float("nan"), float("inf")):
        x[1, 200] = bad
        y = torch.empty(T * k, H, dtype=torch.bfloat16, device=d)
        lib.moe_fp8_experts(shape, T, *w, off, pairs, x, y, ws)
        torch.cuda.synchronize()
        ys.append(y.view(T, k, H))
    rest = torch.arange(T, device=d) != 1
    assert bool(torch.isfinite(ys[0]).all())
    for y in ys[1:]:
        assert bool(torch.isnan(y[1]).all()) and torch.equal(y[rest], ys[0][rest])


@pytest.mark.parametrize("T", [5, 600])
def test_experts_captured_and_shared_workspace(T):
    """Two layers captured into graphs that share one workspace, replayed in turn beside eager calls."""
    rng = np.random.default_rng(77)
    d, (H, I, E, k) = gh.dev(), (256, 128, 4, 2)
    shape = lib.make_shape(H, I, E, k, T, "bf16")
    ws = torch.empty(lib.moe_fp8_experts_workspace_bytes(shape), dtype=torch.uint8, device=d)
    sets = []
    for _ in range(2):
        w = [torch.from_numpy(v).to(d) for v in _layer(rng, H, I, E)]
        x = gh.to_device_x(_x(rng, T, H))
        ids = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).to(d)
        off = torch.empty(E + 1, dtype=torch.int32, device=d)
        pairs, pos = (torch.empty(T * k, dtype=torch.int32, device=d) for _ in range(2))
        lib.moe_permute(shape, T, ids, x, off, pairs, pos, x)
        y = torch.empty(T * k, H, dtype=torch.bfloat16, device=d)
        lib.moe_fp8_experts(shape, T, *w, off, pairs, x, y, ws)
        torch.cuda.synchronize()
        want = y.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.moe_fp8_experts(shape, T, *w, off, pairs, x, y, ws)
        sets.append((g, y, want, (w, x, off, pairs)))  # a graph does not keep its buffers alive
    for i in range(6):
        g, y, want, _ = sets[i % 2]
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
