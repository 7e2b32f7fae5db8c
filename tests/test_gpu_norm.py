"""GPU tests of the RMS norm (mx_rmsnorm, mx_rmsnorm_quantize) and its backward
pass (mx_rmsnorm_backward) against their formulas.

Forward tolerances.  h is one fp32 addition and one rounding, so it equals the
same steps in numpy bit for bit.  rstd: the sum of squares is non-negative, so
its relative error is at most d * 2^-24 for sums of depth d; a thread adds at
most 32 squares (a multiply-add each), the tree over a CTA adds at most 10
levels: d <= 42.  The product with 1 / cols (itself rounded), the addition of
eps and the rounded inverse square root make (42 + 2 + 1) / 2 + 1 < 24 half
steps: |rstd - exact| <= 24 * 2^-24 * exact (a first-order bound; 25 covers
the higher orders).  Given the kernel's rstd, y is two fp32 products and a
rounding, and the codes and scales are the oracle's cast of the fp32 y: all
equal bit for bit.

Backward tolerances, with u = 2^-24, n = h * rstd, a = dy * w and c = mean(a n):
n and a carry one rounding each, their product's sum at most 32 + 10 more and
the product with 1 / cols two, so c is off by at most 46 u mean|a n|.  dx = rstd (a - n c) +
dres: off by at most |rstd| (2 u |a| + 3 u |n c| + 46 u |n| mean|a n|) + 2 u
|dx - dres| + u |dx|, and half a step of the output type.  dweight: n rounds
once, at most ceil(rows / 296) rows are added in turn, then at most 8 groups and
296 parts in any order: (ceil(rows / 296) + 306) u sum|dy n|.
"""
import numpy as np
import pytest
import torch

import mx_independent as ind
from gpu_helpers import dev, first_mismatch, host, to_device
from microscaling_block_scaled_mx_b200 import mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def widen(a):
    """Device or host values as float32 numpy."""
    if isinstance(a, torch.Tensor):
        return a.detach().float().cpu().numpy()
    return a


def make(rows, cols, dtype, seed, spread=2.0):
    g = np.random.default_rng(seed)
    x = (g.standard_normal((rows, cols)) * np.exp2(g.uniform(-spread, spread, (rows, 1)))).astype(np.float32)
    return torch.from_numpy(x).to(dtype).to(dev())


def make_weight(cols, dtype, seed):
    g = np.random.default_rng(seed)
    return torch.from_numpy((1 + 0.2 * g.standard_normal(cols)).astype(np.float32)).to(dtype).to(dev())


def round_to(a32, dtype):
    return torch.from_numpy(np.ascontiguousarray(a32, dtype=np.float32)).to(dtype).float().numpy()


def expected_h(x, residual):
    if residual is None:
        return widen(x)
    return round_to(widen(x) + widen(residual), x.dtype)


def check_rstd(rstd, h, eps):
    want = 1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(1) + eps)
    got = host(rstd).astype(np.float64)
    assert np.all(np.abs(got - want) <= 25 * U * want), np.abs(got / want - 1).max() / U


def y32(h, rstd, w):
    return ((h * host(rstd)[:, None]).astype(np.float32) * widen(w)[None, :]).astype(np.float32)


def same_values(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok].view(np.uint32), want[ok].view(np.uint32))


def same_codes(codes, scales, y, fmt, layout, oracle, rnd="rne", seed=0):
    sl = {"plain": oracle.PLAIN, "mma": oracle.MMA, "mma_x4": oracle.MMA_X4}[layout]
    oc, os_ = oracle.quantize(y, 1, oracle.FORMATS[fmt], rnd=oracle.SR if rnd == "sr" else oracle.RNE, seed=seed,
                              scale_layout=sl, fill=0xAB)
    got = host(codes).reshape(oc.shape)
    assert np.array_equal(got, oc), first_mismatch(got, oc)
    assert np.array_equal(host(scales)[:os_.size], os_)       # padding bytes included: untouched


def filled(rows, cols, fmt, layout):
    u8 = dict(dtype=torch.uint8, device=dev())
    return (torch.full((rows, mx.codes_row_bytes(fmt, cols)), 0xAB, **u8),
            torch.full((max(mx.scales_bytes(layout, rows, cols), 1),), 0xAB, **u8))


SHAPES = [(1, 32), (1, 4096), (3, 64), (130, 96), (64, 1056), (257, 4096), (5, 8192), (4, 8224), (3, 16384),
          (2, 16416), (3, 32768), (1000, 256)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [True, False])
def test_norm(rows, cols, dtype, res):
    x, w = make(rows, cols, dtype, 1), make_weight(cols, dtype, 2)
    r = make(rows, cols, dtype, 3) if res else None
    y, h, rstd = mx.rmsnorm(x, w, 1e-5, residual=r, with_rstd=True)
    eh = expected_h(x, r)
    if res:
        same_values(widen(h), eh)
    else:
        assert h is None
    check_rstd(rstd, eh, 1e-5)
    same_values(widen(y), round_to(y32(eh, rstd, w), dtype))


@pytest.mark.parametrize("rows,cols", [(1, 32), (130, 96), (33, 1056), (200, 4096), (3, 8224), (2, 32768)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m3", "e3m2", "e2m1", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_cast(oracle, rows, cols, fmt, dtype):
    layout = {"e4m3": "mma", "e5m2": "plain", "e2m3": "mma_x4", "e3m2": "mma", "e2m1": "mma_x4", "int8": "plain"}[fmt]
    x, w, r = make(rows, cols, dtype, 4), make_weight(cols, torch.float32, 5), make(rows, cols, dtype, 6)
    codes, scales = filled(rows, cols, fmt, layout)
    out = mx.rmsnorm_quantize(x, w, 1e-6, residual=r, fmt=fmt, scale_layout=layout, with_y=True, with_rstd=True,
                              out=(codes, scales, None, None, None))
    _, _, h, y, rstd = out
    eh = expected_h(x, r)
    same_values(widen(h), eh)
    check_rstd(rstd, eh, 1e-6)
    ey = y32(eh, rstd, w)
    same_values(widen(y), round_to(ey, dtype))
    same_codes(codes, scales, ey, fmt, layout, oracle)
    # without the extras: the same codes
    plain = mx.rmsnorm_quantize(x, w, 1e-6, residual=r, fmt=fmt, scale_layout=layout,
                                out=(*filled(rows, cols, fmt, layout), None, None, None))
    assert plain[3] is None and plain[4] is None
    assert torch.equal(plain[0], codes) and torch.equal(plain[1], scales)


@pytest.mark.parametrize("layout", ["plain", "mma", "mma_x4"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (127, 160), (128, 512), (129, 4096), (300, 2080)])
def test_norm_cast_layouts(oracle, layout, rows, cols):
    x, w = make(rows, cols, torch.bfloat16, 7), make_weight(cols, torch.bfloat16, 8)
    codes, scales = filled(rows, cols, "e4m3", layout)
    out = mx.rmsnorm_quantize(x, w, scale_layout=layout, with_rstd=True, out=(codes, scales, None, None, None))
    assert out[2] is None and out[3] is None
    same_codes(codes, scales, y32(widen(x), out[4], w), "e4m3", layout, oracle)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m3", "e3m2", "e2m1", "int8"])
def test_norm_cast_stochastic(oracle, fmt):
    rows, cols = 70, 1056
    x, w = make(rows, cols, torch.bfloat16, 9), make_weight(cols, torch.bfloat16, 10)
    codes, scales = filled(rows, cols, fmt, "mma")
    seed = 0x123456789ABCDEF
    out = mx.rmsnorm_quantize(x, w, fmt=fmt, rnd="sr", seed=seed, with_rstd=True,
                              out=(codes, scales, None, None, None))
    same_codes(codes, scales, y32(widen(x), out[4], w), fmt, "mma", oracle, rnd="sr", seed=seed)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_rows(oracle, dtype):
    rows, cols = 10, 416
    x = make(rows, cols, torch.float32, 11).cpu()
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 37] = float("inf")
    x[3, 400] = float("-inf")
    x[4] = 1e-40                                    # subnormals: their squares vanish
    x[5] = 3e30                                     # squares overflow: rstd 0
    x[6, 1:] = 0.0
    x[7] = -0.0
    x[8, 64:96] = 0.0                               # a block of zeros
    x = x.to(dtype).to(dev())
    w = make_weight(cols, dtype, 12)
    w[100] = 0.0
    for eps in (0.0, 1e-5):
        codes, scales = filled(rows, cols, "e4m3", "mma")
        _, _, _, y, rstd = mx.rmsnorm_quantize(x, w, eps, with_y=True, with_rstd=True,
                                               out=(codes, scales, None, None, None))
        with np.errstate(all="ignore"):
            ey = y32(widen(x), rstd, w)
            got = host(rstd)
            if eps == 0.0:
                assert np.isinf(got[0]) and np.isinf(got[4]) and np.isinf(got[7])
                assert np.isnan(widen(y)[0]).all()
            else:
                assert got[0] == got[7] and abs(got[0] * np.sqrt(eps) - 1) < 1e-6
                assert not widen(y)[0].any()
            assert np.isnan(got[1]) and got[2] == 0.0 and got[3] == 0.0 and got[5] == 0.0
            same_values(widen(y), round_to(ey, dtype))
            same_codes(codes, scales, ey, "e4m3", "mma", oracle)


def pitched(t, extra):
    full = torch.full((t.shape[0], t.shape[1] + extra), -7.0, dtype=t.dtype, device=t.device)
    full[:, :t.shape[1]] = t
    return full, full[:, :t.shape[1]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pitched_rows(dtype):
    rows, cols = 37, 1056
    x, r, w = make(rows, cols, dtype, 13), make(rows, cols, dtype, 14), make_weight(cols, dtype, 15)
    want = mx.rmsnorm(x, w, residual=r, with_rstd=True)
    _, xv = pitched(x, 8)
    _, rv = pitched(r, 40)
    hf, hv = pitched(torch.zeros_like(x), 16)
    yf, yv = pitched(torch.zeros_like(x), 24)
    y, h, rstd = mx.rmsnorm(xv, w, residual=rv, with_rstd=True, out=(yv, hv, None))
    for a, b in zip((y, h, rstd), want):
        assert torch.equal(a, b)
    assert (hf[:, cols:] == -7).all() and (yf[:, cols:] == -7).all()
    dy, dres = make(rows, cols, dtype, 16), make(rows, cols, dtype, 17)
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    _, dyv = pitched(dy, 8)
    _, drv = pitched(dres, 16)
    xf, dxv = pitched(torch.zeros_like(x), 32)
    dx2, dw2 = mx.rmsnorm_backward(dyv, hv, w, rstd, dres=drv, out=(dxv, None))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and (xf[:, cols:] == -7).all()


def test_in_place():
    rows, cols = 65, 4096
    x, r, w = make(rows, cols, torch.bfloat16, 18), make(rows, cols, torch.bfloat16, 19), make_weight(cols, torch.bfloat16, 20)
    y, h, _ = mx.rmsnorm(x, w, residual=r)
    x1, r1 = x.clone(), r.clone()
    y1, h1, _ = mx.rmsnorm(x1, w, residual=r1, out=(x1, r1, None))        # h over the residual, y over x
    assert torch.equal(y1, y) and torch.equal(h1, h) and h1 is r1 and y1 is x1
    x2 = x.clone()
    _, h2, _ = mx.rmsnorm(x2, w, residual=r, out=(None, x2, None))
    assert torch.equal(h2, h)
    rstd = mx.rmsnorm(h, w, with_rstd=True)[2]
    dy, dres = make(rows, cols, torch.bfloat16, 21), make(rows, cols, torch.bfloat16, 22)
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    for over in (0, 1):
        a = [dy.clone(), dres.clone()]
        dx1, dw1 = mx.rmsnorm_backward(a[0], h, w, rstd, dres=a[1], out=(a[over], None))
        assert torch.equal(dx1, dx) and torch.equal(dw1, dw)


def test_rows_are_independent():
    """A row's result does not depend on the rows beside it."""
    x, w = make(513, 2080, torch.bfloat16, 23), make_weight(2080, torch.bfloat16, 24)
    whole = mx.rmsnorm(x, w, with_rstd=True)
    part = mx.rmsnorm(x[200:203], w, with_rstd=True)
    assert torch.equal(whole[0][200:203], part[0]) and torch.equal(whole[2][200:203], part[2])


def back_inputs(rows, cols, dtype, seed, res):
    h, w = make(rows, cols, dtype, seed), make_weight(cols, dtype, seed + 1)
    dy = make(rows, cols, dtype, seed + 2, spread=1.0)
    dres = make(rows, cols, dtype, seed + 3) if res else None
    return h, w, dy, dres, mx.rmsnorm(h, w, with_rstd=True)[2]


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (130, 96), (333, 1056), (600, 256), (1300, 4096), (9, 8224),
                                       (4, 16416), (3, 32768)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [True, False])
def test_backward(rows, cols, dtype, res):
    h, w, dy, dres, rstd = back_inputs(rows, cols, dtype, 30, res)
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    h6, w6, g6, rs = (widen(t).astype(np.float64) for t in (h, w, dy, rstd))
    rs = rs[:, None]
    n, a = h6 * rs, g6 * w6
    c, c_abs = (a * n).mean(1, keepdims=True), np.abs(a * n).mean(1, keepdims=True)
    core = rs * (a - n * c)
    want = core + (widen(dres).astype(np.float64) if res else 0.0)
    bound = (rs * (2 * np.abs(a) + 3 * np.abs(n * c) + 46 * np.abs(n) * c_abs) + 2 * np.abs(core) + np.abs(want)) * U
    bound = 1.001 * bound + np.abs(want) * HALF[dtype] + 1e-38
    err = np.abs(widen(dx).astype(np.float64) - want)
    assert np.all(err <= bound), (err / bound).max()
    want_w, abs_w = (g6 * n).sum(0), np.abs(g6 * n).sum(0)
    err = np.abs(host(dw).astype(np.float64) - want_w)
    assert np.all(err <= 1.001 * (-(-rows // 296) + 306) * U * abs_w + 1e-38)
    # the same call again: the same bits
    dx2, dw2 = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("rows,cols", [(70, 8224), (150, 16416), (149, 20000), (80, 32768)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_of_wide_rows(rows, cols, dtype):
    """Rows that two or four CTAs share, in uneven pieces, and more rows than run at a time."""
    test_backward(rows, cols, dtype, True)


@pytest.mark.parametrize("cols", [4096, 20000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_in_place_on_a_stream_and_captured(cols, dtype):
    """dx over dy and over dres, off the current stream and in a graph: the same bits."""
    rows = 300
    h, w, dy, dres, rstd = back_inputs(rows, cols, dtype, 31, True)
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    for place in (dy, dres):
        copies = dy.clone(), dres.clone()
        into = copies[0] if place is dy else copies[1]
        ws = mx.rmsnorm_backward_workspace(rows, cols)
        got_w = torch.empty_like(dw)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        mx.rmsnorm_backward(copies[0], h, w, rstd, dres=copies[1], out=(into, got_w), workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(into, dx) and torch.equal(got_w, dw)
    out = torch.empty_like(dx), torch.empty_like(dw)
    ws = mx.rmsnorm_backward_workspace(rows, cols)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):                          # one after the other in the same workspace
            mx.rmsnorm_backward(dy, h, w, rstd, dres=dres, out=out, workspace=ws)
    for t in (*out, ws):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], dx) and torch.equal(out[1], dw)


def test_backward_against_differences():
    """Directional derivatives of the forward formula in fp64.  With step t the
    central difference is off by t^2 / 6 times the third derivative; t = 1e-4
    leaves about 1e-8, and the fp32 gradients about 1e-6 of their size."""
    rows, cols, eps = 4, 96, 1e-5
    g = np.random.default_rng(40)
    h, w = g.standard_normal((rows, cols)).astype(np.float32), (1 + 0.2 * g.standard_normal(cols)).astype(np.float32)
    dy = g.standard_normal((rows, cols)).astype(np.float32)

    def loss(hh, ww):
        return (dy.astype(np.float64) * hh / np.sqrt((hh ** 2).mean(1, keepdims=True) + eps) * ww).sum()

    th, tw = to_device(h), to_device(w)
    rstd = mx.rmsnorm(th, tw, eps, with_rstd=True)[2]
    dx, dw = (host(t).astype(np.float64) for t in mx.rmsnorm_backward(to_device(dy), th, tw, rstd))
    for k in range(6):
        dh, dww, t = g.standard_normal((rows, cols)), g.standard_normal(cols), 1e-4
        num = (loss(h + t * dh, w + t * dww) - loss(h - t * dh, w - t * dww)) / (2 * t)
        got = (dx * dh).sum() + (dw * dww).sum()
        size = np.sqrt((dx ** 2).sum() * (dh ** 2).sum()) + np.sqrt((dw ** 2).sum() * (dww ** 2).sum())
        assert abs(got - num) <= 1e-6 * size, (k, got, num)


def test_backward_special_values():
    rows, cols = 6, 96
    h, w, dy, dres, rstd = back_inputs(rows, cols, torch.float32, 50, True)
    dy[1, 3] = float("nan")
    dy[2] = 0.0
    h[3] = 0.0
    rstd[3] = 316.0
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[[0, 2, 3, 4, 5]]).all()
    assert torch.equal(dx[2], dres[2])
    assert torch.isnan(dw[3]) and torch.isfinite(dw[torch.arange(cols, device=dev()) != 3]).all()


def test_empty():
    w = make_weight(64, torch.bfloat16, 60)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=dev())
    y, h, rstd = mx.rmsnorm(x, w, residual=x, with_rstd=True)
    assert y.shape == (0, 64) and h.shape == (0, 64) and rstd.shape == (0,)
    codes, scales, *_ = mx.rmsnorm_quantize(x, w)
    assert codes.shape == (0, 64)
    dw = torch.full((64,), 5.0, device=dev())
    dx, dw = mx.rmsnorm_backward(x, x, w, rstd, out=(None, dw))
    assert dx.shape == (0, 64) and not dw.any()


def test_graph_and_streams():
    rows, cols = 300, 2080
    x, r, w = make(rows, cols, torch.bfloat16, 61), make(rows, cols, torch.bfloat16, 62), make_weight(cols, torch.bfloat16, 63)
    dy = make(rows, cols, torch.bfloat16, 64)

    def step(stream=None):
        q = mx.rmsnorm_quantize(x, w, residual=r, with_rstd=True, scale_layout="plain", stream=stream)
        return (*q[:3], q[4], *mx.rmsnorm_backward(dy, q[2], w, q[4], dres=r, stream=stream))

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)                                # the stream argument alone
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x2 = make(rows, cols, torch.bfloat16, 65)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    again = [t.clone() for t in out]
    for a, b in zip(again, step()):
        assert torch.equal(a, b)
    assert not torch.equal(again[0], want[0])


DEBUG_CALLS = """
import sys, pickle, torch
sys.path.insert(0, {root!r})
from microscaling_block_scaled_mx_b200 import mx
mx.LIB_PATH = {lib!r}
g = torch.Generator(device="cuda").manual_seed(5)
x = torch.randn(133, 1056, generator=g, device="cuda").bfloat16()
w = torch.ones(1056, device="cuda")
out = []
for fmt in ("e4m3", "e2m3", "e2m1", "int8"):
    for layout in ("plain", "mma", "mma_x4"):
        u8 = dict(dtype=torch.uint8, device="cuda")
        codes = torch.full((133, mx.codes_row_bytes(fmt, 1056)), 0xAB, **u8)
        scales = torch.full((mx.scales_bytes(layout, 133, 1056),), 0xAB, **u8)
        mx.rmsnorm_quantize(x, w, fmt=fmt, scale_layout=layout, out=(codes, scales, None, None, None))
        out += [codes.cpu().numpy(), scales.cpu().numpy()]
torch.cuda.synchronize()
pickle.dump((mx.last_device_status(), out), open({path!r}, "wb"))
"""


def test_debug_build_gives_the_same(tmp_path):
    """The bounds-checking build writes the same bytes and reports nothing."""
    import os
    import pickle
    import subprocess
    import sys

    from microscaling_block_scaled_mx_b200 import build as B
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = []
    for k, lib in enumerate((B.LIB, B.build(debug=True))):
        path = str(tmp_path / f"{k}.pkl")
        r = subprocess.run([sys.executable, "-c", DEBUG_CALLS.format(root=root, lib=lib, path=path)],
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        got.append(pickle.load(open(path, "rb")))
    assert got[0][0] == 0 and got[1][0] == 0
    for a, b in zip(got[0][1], got[1][1]):
        assert np.array_equal(a, b)


def test_offsets_past_32_bits(oracle):
    """More than 2^32 bytes and 2^31 values: the last rows are right."""
    rows, cols = 70000, 32768
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev())
    x[-3:] = make(3, cols, torch.bfloat16, 66)
    w = make_weight(cols, torch.bfloat16, 67)
    codes, scales, _, y, rstd = mx.rmsnorm_quantize(x, w, fmt="e4m3", scale_layout="plain", with_y=True,
                                                    with_rstd=True)
    ey = y32(widen(x[-3:]), rstd[-3:], w)
    same_values(widen(y[-3:]), round_to(ey, torch.bfloat16))
    oc, os_ = oracle.quantize(ey, 1, oracle.E4M3, scale_layout=oracle.PLAIN)
    assert np.array_equal(host(codes[-3:]), oc) and np.array_equal(host(scales[-os_.size:]), os_)
    dx, dw = mx.rmsnorm_backward(y, x, w, rstd, out=(y, None))
    want = mx.rmsnorm_backward(to_device(ind.f32_to_bf16_bits_rne(ey)), x[-3:], w, rstd[-3:])
    assert torch.equal(dx[-3:], want[0])
    # the other rows add zeros: the last three rows fall into parts of their own
    bound = 598 * U * (np.abs(round_to(ey, torch.bfloat16)).astype(np.float64) *
                       np.abs(widen(x[-3:]).astype(np.float64) * host(rstd[-3:])[:, None])).sum(0)
    assert np.all(np.abs(host(dw).astype(np.float64) - host(want[1])) <= 2 * bound + 1e-38)


def test_norm_feeds_the_gemm(oracle):
    """Prefill: h = x + r, y = norm(h) cast to E4M3, then the block-scaled GEMM
    on the codes as written; against the product of the decoded operands."""
    M, N, K = 200, 256, 512
    x, r, w = make(M, K, torch.bfloat16, 70), make(M, K, torch.bfloat16, 71), make_weight(K, torch.bfloat16, 72)
    wt = make(N, K, torch.bfloat16, 73, spread=0.5)
    for layout in ("mma", "mma_x4"):
        codes, scales, h, _, _ = mx.rmsnorm_quantize(x, w, residual=r, scale_layout=layout)
        wc, ws = mx.quantize(wt, 1, "e4m3", scale_layout=layout)
        c = mx.gemm(codes, scales, wc, ws, M, N, K, out_dtype=torch.float32, scale_layout=layout)
        a = mx.dequantize(codes, scales, "e4m3", M, K, scale_layout=layout)
        b = mx.dequantize(wc, ws, "e4m3", N, K, scale_layout=layout)
        a6, b6 = host(a).astype(np.float64), host(b).astype(np.float64)
        assert np.all(np.abs(host(c) - a6 @ b6.T) <= 1e-5 * (np.abs(a6) @ np.abs(b6).T) + 1e-30)
        # the decoded operand is the norm: an E4M3 rounding and the scale's
        # clamp of values above 448 away (at most 1/8 of the value below 512)
        h6 = host(h.float()).astype(np.float64)
        y6 = h6 / np.sqrt((h6 ** 2).mean(1, keepdims=True) + 1e-5) * widen(w).astype(np.float64)
        amax = np.abs(y6).reshape(M, -1, 32).max(-1).repeat(32, 1)
        assert np.all(np.abs(a6 - y6) <= np.maximum(np.abs(y6) * 2.0 ** -3, amax * 2.0 ** -16))
    torch.cuda.synchronize()
    assert mx.last_device_status() == 0
