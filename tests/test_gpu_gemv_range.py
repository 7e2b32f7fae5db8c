"""GPU tests of the largest activations that the 4-bit products' documentation
promises a finite result for, in magnitude: 2^120 with MXFP4 weights, whose
blocks' sums are fp32 before their scale (32 * 6 * 2^120 < 2^128), and
2^116 / K with NVFP4 ones, whose whole sum is fp32 before its domain's scale
(K * 6 * 448 * 2^116 / K < 2^128).  Tolerances are test_gpu_gemv.py's."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev
from microscaling_block_scaled_mx_b200 import mx
from test_gpu_gemv import VALUES, check, lay_out

pytestmark = pytest.mark.gpu


def loud(M, K, top, dtype, seed):
    """Activations up to `top`; the first token is `top` throughout, the second quiet but for one value."""
    g = np.random.default_rng(seed)
    x = g.uniform(-1.0, 1.0, (M, K)) * top
    x[0] = top
    x[1] = g.standard_normal(K)
    x[1, K // 2] = -top
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(dev())


def random_codes(N, K, seed):
    codes = np.random.default_rng(seed).integers(0, 256, (N, K // 2), dtype=np.uint8)
    codes[0] = 0x77                                 # 6 throughout
    codes[1] = 0xFF                                 # -6
    w = np.empty((N, K))
    w[:, 0::2], w[:, 1::2] = VALUES[codes & 15], VALUES[codes >> 4]
    return torch.from_numpy(codes).to(dev()), w


@pytest.mark.parametrize("M,N,K", [(2, 40, 64), (9, 129, 4096), (3, 300, 8192)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mxfp4(M, N, K, dtype):
    codes, w = random_codes(N, K, 1)
    table = np.random.default_rng(2).integers(100, 112, (N, K // 32)).astype(np.uint8)
    w = w * np.repeat(np.exp2(table.astype(np.float64) - 127), 32, axis=1)
    x = loud(M, K, 2.0 ** 120, dtype, 3)
    y = mx.gemv(codes, lay_out(table, "mma"), x, N, K)
    assert torch.isfinite(y).all()
    check(y, x, w)


@pytest.mark.parametrize("M,N,K", [(2, 40, 64), (9, 129, 4096), (3, 300, 8192)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nvfp4(M, N, K, dtype):
    codes, w = random_codes(N, K, 4)
    table = np.random.default_rng(5).integers(1, 0x7F, (N, K // 16)).astype(np.uint8)
    table[:2] = 0x7E                                # 448
    e, m = (table >> 3).astype(np.int64), (table & 7).astype(np.float64)
    d = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.exp2(e - 7.0))
    enc = torch.full((1,), 2.0 ** 20, device=dev())
    x = loud(M, K, 2.0 ** 116 / K, dtype, 6)
    y = mx.gemv_nvfp4((codes, lay_out(table, "mma"), enc), x, N, K)
    assert torch.isfinite(y).all()
    check(y, x, w * np.repeat(d, 16, axis=1) * 2.0 ** -20)
