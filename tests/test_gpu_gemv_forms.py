"""GPU tests of calls of the 4-bit products that are accepted and that
test_gpu_gemv.py does not make: alpha with NVFP4 weights and plain scales at
an odd address.  Tolerances are test_gpu_gemv.py's; alpha over the domain's
scale and the product with it are one rounding each, of half of the 2^-23 that
its bound has four of beside the block's forty."""
import pytest
import torch

from gpu_helpers import dev
from microscaling_block_scaled_mx_b200 import mx
from test_gpu_gemv import activations, check, mx_weights, nv_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("alpha", [-0.37, 1e-3, 48.0])
@pytest.mark.parametrize("M,N,K,domain", [(1, 300, 2080, 0), (3, 129, 528, 32), (16, 200, 1024, 7), (20, 33, 4096, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_alpha_with_nvfp4_weights(alpha, M, N, K, domain, dtype):
    ws, w = nv_weights(N, K, "mma", domain, 1)
    x = activations(M, K, dtype, 2)
    check(mx.gemv_nvfp4(ws, x, N, K, domain_rows=domain, alpha=alpha), x, w, alpha)
    assert not mx.gemv_nvfp4(ws, x, N, K, domain_rows=domain, alpha=0.0).any()


def off_the_word(scales, at):
    buf = torch.full((scales.numel() + 8,), 0xFF, dtype=torch.uint8, device=dev())
    view = buf[at:at + scales.numel()]
    view.copy_(scales)
    return view


@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 129, 4096), (5, 1001, 2176), (9, 300, 8192), (16, 33, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_plain_scales_at_an_odd_address(M, N, K, dtype, at):
    """Whole words of scales (K a multiple of 128) that start off a word: the
    same bits as on one."""
    x = activations(M, K, dtype, 3)
    codes, scales, w = mx_weights(N, K, "plain", 4)
    want = mx.gemv(codes, scales, x, N, K, scale_layout="plain")
    check(want, x, w)
    assert torch.equal(mx.gemv(codes, off_the_word(scales, at), x, N, K, scale_layout="plain"), want)
    (codes, scales, enc), w = nv_weights(N, K, "plain", 32, 5)
    want = mx.gemv_nvfp4((codes, scales, enc), x, N, K, domain_rows=32, scale_layout="plain")
    check(want, x, w)
    got = mx.gemv_nvfp4((codes, off_the_word(scales, at), enc), x, N, K, domain_rows=32, scale_layout="plain")
    assert torch.equal(got, want)


def test_a_batch_of_thousands():
    """More tokens than a wave of CTAs takes; each has the bits that it has alone."""
    M, N, K = 4099, 77, 352
    codes, scales, w = mx_weights(N, K, "mma", 6)
    ws, w_nv = nv_weights(N, K, "mma", 7, 7)
    for dtype in (torch.bfloat16, torch.float32):
        x = activations(M, K, dtype, 8)
        y, y_nv = mx.gemv(codes, scales, x, N, K), mx.gemv_nvfp4(ws, x, N, K, 7)
        check(y, x, w)
        check(y_nv, x, w_nv)
        for i in (0, 2048, 4098):
            assert torch.equal(mx.gemv(codes, scales, x[i:i + 1], N, K), y[i:i + 1])
            assert torch.equal(mx.gemv_nvfp4(ws, x[i:i + 1], N, K, 7), y_nv[i:i + 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_longest_rows(dtype):
    M, N, K = 2, 3, 1 << 24
    codes, scales, w = mx_weights(N, K, "plain", 9)
    x = activations(M, K, dtype, 10)
    y = mx.gemv(codes, scales, x, N, K, scale_layout="plain", out_dtype=torch.float32)
    check(y, x, w)
    assert torch.equal(mx.gemv(codes, scales, x[1:], N, K, scale_layout="plain", out_dtype=torch.float32), y[1:])
