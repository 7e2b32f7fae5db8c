"""GPU tests of the norm's weight gradient (mx_rmsnorm_backward): its bits do not
depend on dres, and tall matrices of every width stay within the sum's error.

Tolerance, with u = 2^-24 and n = h * rstd: n rounds once; a thread adds at
most ceil(rows / 32) rows, a multiply-add each (32 shares of the rows is the
fewest that any width has); then at most 8 groups of a CTA, ten of at most 296
shares in a warp and 32 warps: |dweight - exact| <= (ceil(rows / 32) + 51) u
sum |dy n|, first order (1.001 covers the higher orders).
"""
import pytest
import torch

from gpu_helpers import dev
from microscaling_block_scaled_mx_b200 import mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def inputs(rows, cols, dtype, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    h, dy, dres = (torch.randn((rows, cols), device=dev(), generator=g).to(dtype) for _ in range(3))
    w = (1 + 0.2 * torch.randn(cols, device=dev(), generator=g)).to(dtype)
    return h, dy, dres, w, mx.rmsnorm(h, w, with_rstd=True)[2]


@pytest.mark.parametrize("rows,cols,dtype", [
    (600, 4096, BF16), (600, 10240, BF16), (400, 9248, BF16), (400, 14336, BF16), (400, 14368, BF16),
    (600, 5120, F32), (400, 4640, F32), (333, 7168, F32), (333, 7200, F32), (150, 5120, F32), (40, 10240, BF16),
    (200, 20480, BF16), (200, 20480, F32), (700, 96, F32)])
def test_the_same_with_and_without_dres(rows, cols, dtype):
    h, dy, dres, w, rstd = inputs(rows, cols, dtype, 1)
    with_dres = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)[1]
    without = mx.rmsnorm_backward(dy, h, w, rstd)[1]
    assert torch.equal(with_dres, without)


@pytest.mark.parametrize("rows,cols,dtype", [
    (5000, 32, BF16), (9001, 1056, BF16), (3001, 10240, BF16), (2500, 20480, BF16), (3001, 5120, F32), (2500, 10240, F32),
    (2500, 20480, F32)])
@pytest.mark.parametrize("res", [True, False])
def test_tall(rows, cols, dtype, res):
    h, dy, dres, w, rstd = inputs(rows, cols, dtype, 2)
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres if res else None)
    terms = dy.double() * (h.double() * rstd.double()[:, None])
    err, size = (dw.double() - terms.sum(0)).abs(), terms.abs().sum(0)
    assert torch.all(err <= 1.001 * (-(-rows // 32) + 51) * 2.0 ** -24 * size + 1e-38), (err / size).max()
    # the last rows' gradients, as when they come alone
    last = mx.rmsnorm_backward(dy[-3:], h[-3:], w, rstd[-3:], dres=dres[-3:] if res else None)[0]
    assert torch.equal(dx[-3:], last)
