"""GPU tests of calls of the norm that its alignment and types decide: fp32 rows
on 16-byte boundaries that are not 32-byte ones, plain scales at an odd
address, a weight of another type than the data, stochastic rounding with a
residual.  Alignment changes no bit; the rest is compared with the formulas
under the tolerances of test_gpu_norm.py."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host
from microscaling_block_scaled_mx_b200 import mx
from test_gpu_norm import HALF, U, check_rstd, expected_h, filled, make, make_weight, round_to, same_codes, same_values
from test_gpu_norm import widen, y32

pytestmark = pytest.mark.gpu

GUARD = -7.0


def shifted(t, pitch, offset):
    """t's values with `pitch` elements to a row, `offset` elements into a buffer
    of guards; (buffer, view)."""
    rows, cols = t.shape
    buf = torch.full((offset + rows * pitch + 8,), GUARD, dtype=t.dtype, device=t.device)
    view = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
    view.copy_(t)
    return buf, view


def guards_hold(buf, view):
    left = buf.clone()
    off, (rows, cols), pitch = view.storage_offset(), view.shape, view.stride(0)
    left[off:off + rows * pitch].view(rows, pitch)[:, :cols] = GUARD
    return bool((left == GUARD).all())


@pytest.mark.parametrize("pad,offset", [(4, 0), (0, 4), (4, 4), (12, 4), (8, 4)])
@pytest.mark.parametrize("rows,cols", [(1, 96), (37, 96), (300, 1056), (160, 4096), (5, 8224), (3, 20000)])
def test_fp32_rows_on_16_byte_boundaries(rows, cols, pad, offset):
    x, r = make(rows, cols, torch.float32, 1), make(rows, cols, torch.float32, 2)
    w = make_weight(cols, torch.float32, 3)
    want = mx.rmsnorm(x, w, residual=r, with_rstd=True)
    want_q = mx.rmsnorm_quantize(x, w, residual=r)
    alone = mx.rmsnorm(x, w)[0]
    pitch = cols + pad
    (_, xv), (_, rv) = shifted(x, pitch, offset), shifted(r, cols + 8, 0)
    (hb, hv), (yb, yv) = shifted(torch.zeros_like(x), pitch, offset), shifted(torch.zeros_like(x), pitch, offset)
    y, h, rstd = mx.rmsnorm(xv, w, residual=rv, with_rstd=True, out=(yv, hv, None))
    for a, b in zip((y, h, rstd), want):
        assert torch.equal(a, b)
    assert guards_hold(hb, hv) and guards_hold(yb, yv)
    assert torch.equal(mx.rmsnorm(xv, w)[0], alone)
    codes, scales, h2, _, _ = mx.rmsnorm_quantize(xv, w, residual=rv)
    assert torch.equal(codes, want_q[0]) and torch.equal(h2, want_q[2])
    table = mx.rmsnorm_quantize(x, w, residual=r, scale_layout="plain")[1]
    assert torch.equal(mx.rmsnorm_quantize(xv, w, residual=rv, scale_layout="plain")[1], table)
    # one shifted tensor among aligned ones
    y1, h1, _ = mx.rmsnorm(x, w, residual=r, out=(yv.zero_(), None, None))
    assert torch.equal(y1, want[0]) and torch.equal(h1, want[1]) and guards_hold(yb, yv)
    # h over the residual, y over x
    xb2, xv2 = shifted(x, pitch, offset)
    rb2, rv2 = shifted(r, pitch, offset)
    mx.rmsnorm(xv2, w, residual=rv2, out=(xv2, rv2, None))
    assert torch.equal(xv2, want[0]) and torch.equal(rv2, want[1])
    assert guards_hold(xb2, xv2) and guards_hold(rb2, rv2)
    # the gradient
    dy, dres = make(rows, cols, torch.float32, 4), make(rows, cols, torch.float32, 5)
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    (db, dyv), (_, drv) = shifted(dy, pitch, offset), shifted(dres, pitch, offset)
    dx2, dw2 = mx.rmsnorm_backward(dyv, hv, w, rstd, dres=drv, out=(dyv, None))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and guards_hold(db, dyv)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m3", "e2m1"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (130, 256), (33, 4096), (3, 16384)])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_plain_scales_at_an_odd_address(fmt, rows, cols, at):
    """Whole words of scales (cols a multiple of 128) that start off a word."""
    x, w = make(rows, cols, torch.bfloat16, 6), make_weight(cols, torch.bfloat16, 7)
    want = mx.rmsnorm_quantize(x, w, fmt=fmt, scale_layout="plain")
    n = rows * cols // 32
    buf = torch.full((n + 8,), 0xAB, dtype=torch.uint8, device=dev())
    codes, scales, *_ = mx.rmsnorm_quantize(x, w, fmt=fmt, scale_layout="plain",
                                            out=(None, buf[at:at + n], None, None, None))
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1][:n])
    assert (buf[:at] == 0xAB).all() and (buf[at + n:] == 0xAB).all()


OTHER = {torch.bfloat16: torch.float32, torch.float32: torch.bfloat16}


@pytest.mark.parametrize("rows,cols", [(1, 32), (130, 96), (64, 1056), (9, 4096), (3, 8224), (2, 20000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [True, False])
def test_a_weight_of_the_other_type(oracle, rows, cols, dtype, res):
    x, w = make(rows, cols, dtype, 8), make_weight(cols, OTHER[dtype], 9)
    r = make(rows, cols, dtype, 10) if res else None
    y, h, rstd = mx.rmsnorm(x, w, residual=r, with_rstd=True)
    eh = expected_h(x, r)
    check_rstd(rstd, eh, 1e-5)
    ey = y32(eh, rstd, w)
    same_values(widen(y), round_to(ey, dtype))
    codes, scales = filled(rows, cols, "e2m1", "mma")
    mx.rmsnorm_quantize(x, w, residual=r, fmt="e2m1", out=(codes, scales, None, None, None))
    same_codes(codes, scales, ey, "e2m1", "mma", oracle)
    # dx and dweight, with the bounds that test_gpu_norm.py derives
    dy, dres = make(rows, cols, dtype, 11, spread=1.0), make(rows, cols, dtype, 12) if res else None
    hh = x if h is None else h
    dx, dw = mx.rmsnorm_backward(dy, hh, w, rstd, dres=dres)
    assert dx.dtype is dtype and dw.dtype is torch.float32
    h6, w6, g6, rs = (widen(t).astype(np.float64) for t in (hh, w, dy, rstd))
    rs = rs[:, None]
    n, a = h6 * rs, g6 * w6
    c, c_abs = (a * n).mean(1, keepdims=True), np.abs(a * n).mean(1, keepdims=True)
    core = rs * (a - n * c)
    want = core + (widen(dres).astype(np.float64) if res else 0.0)
    bound = (rs * (2 * np.abs(a) + 3 * np.abs(n * c) + 46 * np.abs(n) * c_abs) + 2 * np.abs(core) + np.abs(want)) * U
    bound = 1.001 * bound + np.abs(want) * HALF[dtype] + 1e-38
    err = np.abs(widen(dx).astype(np.float64) - want)
    assert np.all(err <= bound), (err / bound).max()
    err = np.abs(host(dw).astype(np.float64) - (g6 * n).sum(0))
    assert np.all(err <= 1.001 * (-(-rows // 32) + 51) * U * np.abs(g6 * n).sum(0) + 1e-38)


@pytest.mark.parametrize("layout", ["plain", "mma", "mma_x4"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m3", "e3m2", "e2m1", "int8"])
@pytest.mark.parametrize("rows,cols,dtype", [(130, 1056, torch.float32), (5, 8224, torch.float32), (200, 512, torch.bfloat16),
                                             (3, 16416, torch.bfloat16)])
def test_stochastic_rounding_with_a_residual(oracle, layout, fmt, rows, cols, dtype):
    x, r, w = make(rows, cols, dtype, 13), make(rows, cols, dtype, 14), make_weight(cols, dtype, 15)
    codes, scales = filled(rows, cols, fmt, layout)
    seed = 0xFEDCBA9876543210
    _, _, h, y, rstd = mx.rmsnorm_quantize(x, w, residual=r, fmt=fmt, rnd="sr", seed=seed, scale_layout=layout,
                                           with_y=True, with_rstd=True, out=(codes, scales, None, None, None))
    eh = expected_h(x, r)
    same_values(widen(h), eh)
    ey = y32(eh, rstd, w)
    same_values(widen(y), round_to(ey, dtype))
    same_codes(codes, scales, ey, fmt, layout, oracle, rnd="sr", seed=seed)
