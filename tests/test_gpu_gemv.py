"""GPU tests of the products of a few tokens with 4-bit weights (mx_gemv,
mx_gemv_nvfp4) against the product of the exactly decoded weights in fp64.

Tolerance: products of a code with an activation are exact; a block's sum of
32 (or 16) of them is off by at most 40 * 2^-23 of the sum of their
magnitudes, however it is added (tensor cores may truncate instead of round),
and the K / 32 blocks' sums are added in fp32, 2^-23 each: |y - exact| <=
(44 + K / 32) * 2^-23 * |alpha| sum |x w| + half a step of the output type.
Where every partial sum is exact in fp32 (small integers, equal scales), the
result has to be exact.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host
from microscaling_block_scaled_mx_b200 import mx

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
VALUES = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def f64(t):
    return t.detach().double().cpu().numpy()


def activations(M, K, dtype, seed):
    g = np.random.default_rng(seed)
    return torch.from_numpy((g.standard_normal((M, K)) * np.exp2(g.uniform(-3, 3, (M, 1)))).astype(np.float32)
                            ).to(dtype).to(dev())


def mx_weights(N, K, layout, seed, scale_lo=118, scale_hi=130):
    """Random codes and scales: (codes, scales, decoded fp64)."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    table = g.integers(scale_lo, scale_hi + 1, (N, K // 32)).astype(np.uint8)
    w = np.empty((N, K))
    w[:, 0::2], w[:, 1::2] = VALUES[codes & 15], VALUES[codes >> 4]
    w = w * np.repeat(np.exp2(table.astype(np.float64) - 127), 32, axis=1)
    return torch.from_numpy(codes).to(dev()), lay_out(table, layout), w


def nv_weights(N, K, layout, domain, seed):
    g = np.random.default_rng(seed)
    codes = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    table = g.integers(0, 0x7F, (N, K // 16)).astype(np.uint8)          # every finite positive E4M3 value
    e, m = (table >> 3).astype(np.int64), (table & 7).astype(np.float64)
    d = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.exp2(e - 7.0))
    lines = domain or N
    enc = np.exp2(g.uniform(-4, 4, -(-N // lines))).astype(np.float32)
    w = np.empty((N, K))
    w[:, 0::2], w[:, 1::2] = VALUES[codes & 15], VALUES[codes >> 4]
    w = w * np.repeat(d, 16, axis=1) / np.repeat(enc.astype(np.float64), lines)[:N, None]
    return (torch.from_numpy(codes).to(dev()), lay_out(table, layout), torch.from_numpy(enc).to(dev())), w


def lay_out(table, layout):
    """A table of scale bytes in a layout; the padding is 0xFF (NaN in both kinds of scale)."""
    N, KB = table.shape
    if layout == "plain":
        flat = table.reshape(-1)
    else:
        ro, kb = (N + 127) // 128 * 128, (KB + 3) // 4 * 4
        full = np.full((ro, kb), 0xFF, np.uint8)
        full[:N, :KB] = table
        atoms = full.reshape(ro // 128, 4, 32, kb // 4, 4).transpose(0, 3, 2, 1, 4).reshape(-1, 512)
        flat = (np.repeat(atoms, 4, axis=0) if layout == "mma_x4" else atoms).reshape(-1)
    return torch.from_numpy(np.ascontiguousarray(flat)).to(dev())


def check(y, x, w, alpha=1.0):
    K = w.shape[1]
    want = alpha * (f64(x) @ w.T)
    size = abs(alpha) * (np.abs(f64(x)) @ np.abs(w).T)
    err = np.abs(f64(y) - want)
    bound = (44 + K / 32) * 2.0 ** -23 * size
    bound = bound + (np.abs(want) + bound) * HALF[y.dtype] + 1e-38
    assert np.all(err <= bound), (err / bound).max()


SIZES = [(1, 1, 32), (1, 7, 64), (2, 128, 128), (3, 100, 160), (1, 129, 4096), (5, 1001, 2080), (8, 256, 1024),
         (9, 130, 288), (16, 384, 512), (17, 65, 992), (33, 200, 256), (1, 4096, 4096), (4, 33, 14336)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("layout", ["plain", "mma", "mma_x4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemv(M, N, K, layout, dtype):
    codes, scales, w = mx_weights(N, K, layout, 1)
    x = activations(M, K, dtype, 2)
    y = mx.gemv(codes, scales, x, N, K, scale_layout=layout)
    assert y.dtype is dtype and y.shape == (M, N)
    check(y, x, w)
    assert torch.equal(y, mx.gemv(codes, scales, x, N, K, scale_layout=layout))


@pytest.mark.parametrize("M,N,K", [*SIZES, (1, 50, 16), (3, 200, 48), (7, 129, 2064)])
@pytest.mark.parametrize("layout", ["plain", "mma", "mma_x4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemv_nvfp4(M, N, K, layout, dtype):
    domain = {0: 0, 1: 32, 2: 7}[(M + N) % 3]
    ws, w = nv_weights(N, K, layout, domain, 3)
    x = activations(M, K, dtype, 4)
    y = mx.gemv_nvfp4(ws, x, N, K, domain_rows=domain, scale_layout=layout)
    assert y.dtype is dtype and y.shape == (M, N)
    check(y, x, w)


@pytest.mark.parametrize("M,N,K", [(1, 300, 2080), (6, 129, 4096), (16, 200, 544)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_exact_sums(M, N, K, dtype, out_dtype):
    """Whole activations below 16 and one scale: every partial sum is a multiple
    of half the scale below 2^21 of them, exact in fp32 in any order."""
    codes, scales, w = mx_weights(N, K, "mma", 5, scale_lo=121, scale_hi=121)
    x = torch.from_numpy(np.random.default_rng(6).integers(-15, 16, (M, K)).astype(np.float32)).to(dtype).to(dev())
    y = mx.gemv(codes, scales, x, N, K, alpha=0.5, out_dtype=out_dtype)
    want = torch.from_numpy(0.5 * (f64(x) @ w.T)).to(out_dtype)
    assert torch.equal(y.cpu(), want)


def test_tokens_are_independent():
    """A token's result does not depend on the tokens beside it, nor on how many there are."""
    N, K = 260, 1056
    codes, scales, _ = mx_weights(N, K, "mma", 7)
    ws, _ = nv_weights(N, K, "mma", 32, 8)
    for dtype in (torch.bfloat16, torch.float32):
        x = activations(20, K, dtype, 9)
        whole, whole_nv = mx.gemv(codes, scales, x, N, K), mx.gemv_nvfp4(ws, x, N, K, 32)
        for a, b in ((0, 1), (3, 4), (7, 15), (19, 20), (0, 16)):
            assert torch.equal(mx.gemv(codes, scales, x[a:b], N, K), whole[a:b])
            assert torch.equal(mx.gemv_nvfp4(ws, x[a:b], N, K, 32), whole_nv[a:b])


@pytest.mark.parametrize("N,K", [(300, 8192), (4100, 4096), (40, 14336)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_batch_of_any_size_gives_the_same(N, K, dtype):
    """The work is cut differently for one token and for sixteen, the sums are not;
    and a token whose neighbours need bf16 products keeps its bits."""
    codes, scales, _ = mx_weights(N, K, "mma", 40)
    ws, _ = nv_weights(N, K, "mma_x4", 0, 41)
    x = activations(24, K, dtype, 42)
    x[5, 3] = 5000.0                                # past what fp16 takes, in the first slice
    x[17, K - 1] = 1e-12                            # below it, in the last
    x[20] *= 2.0 ** -60
    whole = mx.gemv(codes, scales, x, N, K), mx.gemv_nvfp4(ws, x, N, K, scale_layout="mma_x4")
    for a, b in ((0, 1), (4, 5), (5, 6), (16, 18), (17, 18), (0, 8), (8, 24), (20, 21)):
        assert torch.equal(mx.gemv(codes, scales, x[a:b], N, K), whole[0][a:b]), (a, b)
        assert torch.equal(mx.gemv_nvfp4(ws, x[a:b], N, K, scale_layout="mma_x4"), whole[1][a:b]), (a, b)


@pytest.mark.parametrize("M", [1, 9])
def test_more_rows_than_one_pass(M):
    N, K = 70001, 96
    codes, scales, w = mx_weights(N, K, "mma", 43)
    x = activations(M, K, torch.bfloat16, 44)
    check(mx.gemv(codes, scales, x, N, K), x, w)
    codes, scales, w = mx_weights(N, K, "plain", 45)
    check(mx.gemv(codes, scales, x, N, K, scale_layout="plain"), x, w)


def test_calls_back_to_back():
    """A chain of calls, each reading what the one before wrote, with other work
    between them, as the same calls one at a time."""
    N = K = 2048
    codes, scales, _ = mx_weights(N, K, "mma", 46, 114, 120)
    ws, _ = nv_weights(N, K, "mma", 0, 47)
    gamma = torch.ones(K, device=dev())
    x = activations(2, K, torch.bfloat16, 48)

    def chain(pause):
        h, y = x.clone(), None
        for k in range(12):
            y, h, _ = mx.rmsnorm(h, gamma, residual=h if y is None else y)
            pause()
            y = mx.gemv(codes, scales, y, N, K) if k % 2 else mx.gemv_nvfp4(ws, y, N, K)
            pause()
            if k % 3 == 0:
                y = y * 0.5
                pause()
        return h, y

    want = chain(torch.cuda.synchronize)
    for _ in range(20):
        got = chain(lambda: None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(lambda: None)
    for _ in range(5):
        graph.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_streams_at_once():
    """Calls on two streams at a time, weights shared."""
    N, K = 4096, 2048
    codes, scales, _ = mx_weights(N, K, "mma", 49)
    xs = [activations(3, K, torch.bfloat16, 50 + i) for i in range(2)]
    want = [mx.gemv(codes, scales, x, N, K) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            got[i].append(mx.gemv(codes, scales, xs[i], N, K, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


FIRST_IN_A_GRAPH = """
import sys, torch
sys.path.insert(0, {root!r})
from microscaling_block_scaled_mx_b200 import mx
d = dict(device="cuda")
codes = torch.full((256, 512), 0x22, dtype=torch.uint8, **d)
scales = torch.full((mx.scales_bytes("mma", 256, 1024),), 127, dtype=torch.uint8, **d)
x, w = torch.ones(2, 1024, **d).bfloat16(), torch.ones(1024, **d)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, h, rstd = mx.rmsnorm(x, w, 0.0, residual=x, with_rstd=True)
    q = mx.rmsnorm_quantize(x, w)
    out = mx.gemv(codes, scales, y, 256, 1024)
    dx, dw = mx.rmsnorm_backward(y, h, w, rstd)
graph.replay()
torch.cuda.synchronize()
assert (out == 1024).all() and (h == 2).all() and (dw == 2).all()
"""


def test_first_call_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_layouts_agree():
    N, K = 300, 1184
    x = activations(3, K, torch.bfloat16, 10)
    ys = [mx.gemv(*mx_weights(N, K, sl, 11)[:2], x, N, K, scale_layout=sl) for sl in ("plain", "mma", "mma_x4")]
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_values(dtype):
    M, N, K = 3, 140, 256
    codes, _, w = mx_weights(N, K, "plain", 12, 127, 127)
    g = np.random.default_rng(13)
    table = g.integers(120, 130, (N, K // 32)).astype(np.uint8)
    table[5, 2] = 0xFF                              # a NaN block
    table[6] = 0                                    # 2^-127 throughout
    table[7, 3] = 254                               # 2^127
    with np.errstate(all="ignore"):
        factor = np.where(table == 0xFF, np.nan, np.exp2(table.astype(np.float64) - 127))
    w = w * np.repeat(factor, 32, axis=1)
    x = activations(M, K, dtype, 14)
    x[:, 96:128] *= 2.0 ** -20                      # the 2^127 block stays finite
    x[1, 40] = 0.0
    y = mx.gemv(codes, lay_out(table, "mma"), x, N, K, out_dtype=torch.float32)
    assert torch.isnan(y[:, 5]).all()
    fine = np.arange(N) != 5
    want, size = f64(x) @ w.T, np.abs(f64(x)) @ np.abs(w).T
    err = np.abs(f64(y) - want)[:, fine]
    # row 6: products with 2^-127 are subnormal, one rounding of at most 2^-150 a block
    assert np.all(err <= ((44 + K / 32) * 2.0 ** -23 * size)[:, fine] + 16 * 2.0 ** -149)
    x[1, 40] = float("inf")
    x[2, 41] = float("nan")
    y = mx.gemv(codes, lay_out(table, "mma"), x, N, K, out_dtype=torch.float32)
    with np.errstate(all="ignore"):
        ref = f64(x) @ w.T
    assert torch.isnan(y[2]).all() and torch.isfinite(y[0, torch.arange(N, device=dev()) != 5]).all()
    got = f64(y)[1]
    assert np.array_equal(np.isnan(got), np.isnan(ref[1])) and np.array_equal(np.isinf(got), np.isinf(ref[1]))
    inf = np.isinf(ref[1])
    assert np.array_equal(np.sign(got[inf]), np.sign(ref[1][inf]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wide_range_of_activations(dtype):
    """Activations from the smallest normals to the largest, one loud value a
    token whose weight is zero: the quiet ones still count."""
    N, K = 130, 512
    g = np.random.default_rng(15)
    codes, scales, w = mx_weights(N, K, "mma", 16, 127, 127)
    host_codes = host(codes).copy()
    host_codes[:, 0] &= 0xF0
    codes = torch.from_numpy(host_codes).to(dev())
    w[:, 0] = 0.0
    x = np.stack([g.standard_normal(K) * s for s in (1e-30, 1e30, 1.0, 2.0 ** -120)]).astype(np.float32)
    x[:, 0] = [3e38, 1e-38, -3e38, 1.0]
    t = torch.from_numpy(x).to(dtype).to(dev())
    y = mx.gemv(codes, scales, t, N, K, out_dtype=torch.float32)
    want, size = f64(t) @ w.T, np.abs(f64(t)) @ np.abs(w).T
    assert np.all(np.abs(f64(y) - want) <= (44 + K / 32) * 2.0 ** -23 * size + K * 2.0 ** -133)


def test_nvfp4_special_scales():
    N, K = 130, 128
    g = np.random.default_rng(17)
    (codes, _, enc), _ = nv_weights(N, K, "plain", 0, 18)
    table = g.integers(0, 0x7F, (N, K // 16)).astype(np.uint8)
    table[3, 1] = 0x7F
    table[4] = 0
    x = activations(2, K, torch.bfloat16, 19)
    y = mx.gemv_nvfp4((codes, lay_out(table, "mma"), enc), x, N, K)
    assert torch.isnan(y[:, 3]).all() and not y[:, 4].any()
    keep = torch.arange(N, device=dev()) != 3
    assert torch.isfinite(y[:, keep]).all()


def test_against_the_casts(oracle):
    """Weights as quantize and quantize_nvfp4 write them, against the oracle's decode."""
    N, K = 384, 1024
    wt = activations(N, K, torch.bfloat16, 20)
    x = activations(2, K, torch.bfloat16, 21)
    for layout, sl in (("mma", oracle.MMA), ("mma_x4", oracle.MMA_X4)):
        codes, scales = mx.quantize(wt, 1, "e2m1", scale_layout=layout)
        w = oracle.dequantize(host(codes), host(scales), oracle.E2M1, N, K, sl)
        check(mx.gemv(codes, scales, x, N, K, scale_layout=layout, alpha=-2.0), x, w, -2.0)
    ws = mx.quantize_nvfp4(wt, 128)
    w = oracle.nvfp4_dequantize(host(ws[0]), host(ws[1]), host(ws[2]), N, K, 128, oracle.MMA)
    check(mx.gemv_nvfp4(ws, x, N, K, domain_rows=128), x, w)


def test_pitched_and_untouched():
    M, N, K = 5, 201, 320
    codes, scales, _ = mx_weights(N, K, "mma", 22)
    x = activations(M, K, torch.bfloat16, 23)
    want = mx.gemv(codes, scales, x, N, K)
    xf = torch.full((M, K + 24), 9.0, dtype=torch.bfloat16, device=dev())
    xf[:, :K] = x
    yf = torch.full((M + 2, N + 5), -7.0, dtype=torch.bfloat16, device=dev())
    y = mx.gemv(codes, scales, xf[:, :K], N, K, out=yf[1:M + 1, 3:N + 3])
    assert torch.equal(y, want)
    yf[1:M + 1, 3:N + 3] = -7.0
    assert (yf == -7.0).all()


def test_empty():
    codes, scales, _ = mx_weights(64, 64, "plain", 24)
    assert mx.gemv(codes, scales, torch.empty((0, 64), device=dev()), 64, 64, scale_layout="plain").shape == (0, 64)
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    assert mx.gemv(none, none, torch.empty((2, 64), device=dev()), 0, 64).shape == (2, 0)
    out = torch.full((2, 64), 3.0, device=dev())
    assert not mx.gemv(none, none, torch.empty((2, 0), device=dev()), 64, 0, out=out).any()


def test_graph_and_streams():
    N, K = 1000, 2048
    codes, scales, _ = mx_weights(N, K, "mma", 25)
    ws, _ = nv_weights(N, K, "mma", 32, 26)
    x = activations(1, K, torch.bfloat16, 27)
    side = torch.cuda.Stream()
    want = (mx.gemv(codes, scales, x, N, K), mx.gemv_nvfp4(ws, x, N, K, 32))
    torch.cuda.synchronize()
    got = (mx.gemv(codes, scales, x, N, K, stream=side), mx.gemv_nvfp4(ws, x, N, K, 32, stream=side))
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (mx.gemv(codes, scales, x, N, K), mx.gemv_nvfp4(ws, x, N, K, 32))
    x.copy_(activations(1, K, torch.bfloat16, 28))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], mx.gemv(codes, scales, x, N, K)) and not torch.equal(out[0], want[0])
    assert torch.equal(out[1], mx.gemv_nvfp4(ws, x, N, K, 32))


def test_offsets_past_32_bits():
    """More than 2^32 bytes of codes: the last rows are right."""
    N, K = 33000, 262144
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=dev())
    scales = torch.full((N * (K // 32),), 127, dtype=torch.uint8, device=dev())
    tail, _, w = mx_weights(3, K, "plain", 29, 127, 127)
    codes[-3:] = tail
    x = activations(1, K, torch.bfloat16, 30)
    y = mx.gemv(codes, scales, x, N, K, scale_layout="plain", out_dtype=torch.float32)
    check(y[:, -3:], x, w)
    assert not y[:, :-3].any()


def test_a_decoding_step():
    """norm with the residual, then a product with 4-bit weights on its result, as one
    token passes them; the same weights serve the GEMM of a longer prompt."""
    K, N = 1024, 384
    g = np.random.default_rng(31)
    x, r = activations(3, K, torch.bfloat16, 32), activations(3, K, torch.bfloat16, 33)
    gamma = torch.from_numpy((1 + 0.1 * g.standard_normal(K)).astype(np.float32)).to(dev())
    wc, wsc = mx.quantize(activations(N, K, torch.bfloat16, 34), 1, "e2m1")
    y, h, _ = mx.rmsnorm(x, gamma, residual=r)
    out = mx.gemv(wc, wsc, y, N, K)
    w = f64(mx.dequantize(wc, wsc, "e2m1", N, K))
    check(out, y, w)
    h6 = f64(x) + f64(r)
    assert np.all(np.abs(f64(h) - h6) <= np.abs(h6) * (2.0 ** -8 + 2.0 ** -23))
    h6 = f64(h)
    y6 = h6 / np.sqrt((h6 ** 2).mean(1, keepdims=True) + 1e-5) * f64(gamma)
    assert np.all(np.abs(f64(y) - y6) <= np.abs(y6) * (2.0 ** -8 + 2.0 ** -18))
    # the prompt: the same norm cast to E2M1 against the same weight buffers
    codes, scales, *_ = mx.rmsnorm_quantize(x, gamma, residual=r, fmt="e2m1")
    c = mx.gemm(codes, scales, wc, wsc, 3, N, K, fa="e2m1", out_dtype=torch.float32)
    a = f64(mx.dequantize(codes, scales, "e2m1", 3, K))
    assert np.all(np.abs(f64(c) - a @ w.T) <= 1e-5 * (np.abs(a) @ np.abs(w).T) + 1e-30)
    torch.cuda.synchronize()
    assert mx.last_device_status() == 0


@pytest.mark.parametrize("N", [28416, 19000])
def test_two_and_three_parts_of_k(N):
    """Sizes whose K is cut in two or three: sixteen tokens, whose two parts a
    cluster shares, have the bits of one, which is checked against the product."""
    K = 2304
    g = torch.Generator(device=dev()).manual_seed(50)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev(), generator=g)
    scales = torch.randint(118, 130, (N, K // 32), dtype=torch.uint8, device=dev(), generator=g)
    x = activations(16, K, torch.bfloat16, 51)
    y = mx.gemv(codes, scales, x, N, K, scale_layout="plain", out_dtype=torch.float32)
    assert all(torch.equal(y[i:i + 1], mx.gemv(codes, scales, x[i:i + 1], N, K, scale_layout="plain",
                                               out_dtype=torch.float32)) for i in (0, 7, 15))
    pick = [0, 1, 127, 128, N // 2, N - 130, N - 1]
    c, s = codes[pick].cpu().numpy(), scales[pick].cpu().numpy()
    w = np.empty((len(pick), K))
    w[:, 0::2], w[:, 1::2] = VALUES[c & 15], VALUES[c >> 4]
    check(y[:, pick], x, w * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=1))


@pytest.mark.parametrize("M,N,K,dtype", [
    (3, 1, 32, torch.float32), (3, 1, 512, torch.float32),                # one tile, warps that only stage
    (3, 17, 2080, torch.float32), (3, 1, 65536, torch.float32),           # a cluster of eight, one and two windows
    (16, 33, 4096, torch.bfloat16), (16, 1000, 8192, torch.bfloat16), (8, 777, 1056, torch.bfloat16),
    (3, 300, 2080, torch.float32), (8, 300, 28672, torch.float32),        # a cluster of four
    (8, 1000, 8192, torch.float32), (8, 2300, 2080, torch.float32), (8, 4100, 28672, torch.bfloat16),
    (8, 20000, 2080, torch.float32), (8, 41000, 4096, torch.float32),     # whole rows to a warp, more passes than one
    (3, 70000, 4096, torch.bfloat16), (30, 128, 131072, torch.bfloat16)])
def test_forms_of_the_launch(M, N, K, dtype):
    """Every way in which the work is cut over warps, clusters and windows: the
    first and last token as when they come alone, rows against the product."""
    g = torch.Generator(device=dev()).manual_seed(60)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev(), generator=g)
    scales = torch.randint(118, 130, (N, K // 32), dtype=torch.uint8, device=dev(), generator=g)
    x = activations(M, K, dtype, 61)
    x[M - 1, K // 2] = 3e4                          # a slice of the last token past fp16's range
    y = mx.gemv(codes, scales, x, N, K, scale_layout="plain", out_dtype=torch.float32)
    for i in (0, M - 1):
        assert torch.equal(y[i:i + 1], mx.gemv(codes, scales, x[i:i + 1], N, K, scale_layout="plain",
                                               out_dtype=torch.float32))
    pick = sorted({0, 1 % N, N // 3, N // 2, max(N - 17, 0), N - 1})
    c, s = codes[pick].cpu().numpy(), scales[pick].cpu().numpy()
    w = np.empty((len(pick), K))
    w[:, 0::2], w[:, 1::2] = VALUES[c & 15], VALUES[c >> 4]
    check(y[:, pick], x, w * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=1))
