"""What the norm and the 4-bit products refuse, without a GPU: the C entry
points' status codes before anything is launched, and the binding's checks."""
import pytest
import torch


@pytest.fixture(scope="module")
def mx():
    import ctypes

    from microscaling_block_scaled_mx_b200 import build, mx as m
    build.build()
    L = m.lib()                         # the binding itself calls the packed forms
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.mx_rmsnorm.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, i32, f32, vp, i64, vp, i64, vp, vp]
    L.mx_rmsnorm_quantize.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, i32, f32, i32, i32, ctypes.c_uint64, vp,
                                      i64, vp, i64, vp, vp, vp, i32, vp]
    L.mx_rmsnorm_backward.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, i32, vp, vp, i64, vp, i64, vp, vp,
                                      ctypes.c_size_t, vp]
    L.mx_gemv.argtypes = [vp, vp, i32, i32, vp, i32, i64, i64, i64, i64, f32, vp, i32, i64, vp]
    L.mx_gemv_nvfp4.argtypes = [vp, vp, vp, i64, i32, vp, i32, i64, i64, i64, i64, f32, vp, i32, i64, vp]
    return m


def _n(mx, x=16, xdt=1, rows=4, cols=64, ldx=64, res=None, ldr=64, w=16, wdt=1, eps=1e-5, h=None, ldh=64, y=16,
       ldy=64, rstd=None):
    return mx.lib().mx_rmsnorm(x, xdt, rows, cols, ldx, res, ldr, w, wdt, eps, h, ldh, y, ldy, rstd, None)


def test_rmsnorm_refusals(mx):
    assert _n(mx, xdt=2) == -1 and _n(mx, wdt=-1) == -1
    assert _n(mx, rows=-1) == -1 and _n(mx, cols=-32) == -1
    assert _n(mx, cols=48) == -3
    assert _n(mx, eps=-1e-5) == -1 and _n(mx, eps=float("nan")) == -1 and _n(mx, eps=float("inf")) == -1
    assert _n(mx, rows=0, x=None, w=None, y=None) == 0 and _n(mx, cols=0, x=None) == 0
    assert _n(mx, x=None) == -1 and _n(mx, w=None) == -1 and _n(mx, y=None) == -1
    assert _n(mx, res=16) == -1 and _n(mx, h=16) == -1          # residual and h go together
    assert _n(mx, ldx=32) == -1 and _n(mx, ldy=32) == -1
    assert _n(mx, res=16, h=16, ldr=32) == -1 and _n(mx, res=16, h=16, ldh=32) == -1
    assert _n(mx, x=8) == -2 and _n(mx, y=24) == -2 and _n(mx, w=8) == -2 and _n(mx, rstd=2) == -2
    assert _n(mx, ldx=68) == -2 and _n(mx, xdt=0, ldx=66) == -2
    assert _n(mx, res=8, h=16) == -2 and _n(mx, res=16, h=8) == -2
    assert _n(mx, cols=32800, ldx=32800, ldy=32800) == -4
    assert _n(mx, rows=1 << 31) == -4


def _q(mx, rows=4, cols=64, ld=64, fmt=0, rnd=0, sl=1, codes=16, scales=16, y=None, res=None, h=None):
    return mx.lib().mx_rmsnorm_quantize(16, 1, rows, cols, ld, res, ld, 16, 1, 1e-5, fmt, rnd, 0, h, ld, y, ld, None,
                                        codes, scales, sl, None)


def test_rmsnorm_quantize_refusals(mx):
    assert _q(mx, fmt=6) == -1 and _q(mx, rnd=2) == -1 and _q(mx, sl=3) == -1
    assert _q(mx, codes=None) == -1 and _q(mx, scales=None) == -1
    assert _q(mx, codes=24) == -2 and _q(mx, y=8) == -2
    assert _q(mx, rows=0, codes=None, scales=None) == 0
    assert _q(mx, res=16) == -1
    assert _q(mx, rows=1 << 30, cols=32, ld=32, rnd=1) == -5              # 2^35 values
    assert _q(mx, rows=1 << 30, cols=256, ld=256, sl=0) == -4             # 8 GiB of scales


def _b(mx, dy=16, xdt=1, rows=4, cols=64, ld=64, h=16, w=16, rstd=16, dres=None, ldr=64, dx=16, lddx=64, dw=16,
       ws=16, n=None):
    L = mx.lib()
    if n is None:
        n = L.mx_rmsnorm_backward_workspace_bytes(max(rows, 0), 64)
    return L.mx_rmsnorm_backward(dy, xdt, rows, cols, ld, h, ld, w, 1, rstd, dres, ldr, dx, lddx, dw, ws, n, None)


def test_rmsnorm_backward_refusals(mx):
    L = mx.lib()
    assert L.mx_rmsnorm_backward_workspace_bytes(3, 64) == 3 * 64 * 4
    assert L.mx_rmsnorm_backward_workspace_bytes(10 ** 9, 4096) == 296 * 4096 * 4
    assert L.mx_rmsnorm_backward_workspace_bytes(-1, 64) == 0 and L.mx_rmsnorm_backward_workspace_bytes(3, 33) == 0
    assert _b(mx, xdt=5) == -1 and _b(mx, rows=-1) == -1 and _b(mx, cols=40) == -3
    assert _b(mx, cols=0, dy=None, dw=None) == 0
    for name in ("dy", "h", "w", "rstd", "dx", "dw", "ws"):
        assert _b(mx, **{name: None}) == -1, name
    assert _b(mx, n=3 * 64 * 4) == -1                                    # workspace too small
    assert _b(mx, ld=32) == -1 and _b(mx, lddx=32) == -1 and _b(mx, dres=16, ldr=32) == -1
    assert _b(mx, dy=8) == -2 and _b(mx, dx=8) == -2 and _b(mx, ws=8) == -2 and _b(mx, rstd=2) == -2
    assert _b(mx, dw=2) == -2 and _b(mx, dres=8) == -2 and _b(mx, ld=68) == -2
    assert _b(mx, cols=32800, ld=32800, lddx=32800) == -4


def _v(mx, codes=16, scales=16, fw=4, sl=1, x=16, xdt=1, ldx=256, M=1, N=64, K=256, y=16, ydt=1, ldy=64):
    return mx.lib().mx_gemv(codes, scales, fw, sl, x, xdt, ldx, M, N, K, 1.0, y, ydt, ldy, None)


def test_gemv_refusals(mx):
    assert _v(mx, fw=7) == -1 and _v(mx, fw=0) == -4 and _v(mx, fw=5) == -4
    assert _v(mx, xdt=2) == -1 and _v(mx, ydt=2) == -1 and _v(mx, sl=3) == -1
    assert _v(mx, M=-1) == -1 and _v(mx, N=-1) == -1 and _v(mx, K=-32) == -1
    assert _v(mx, K=48) == -3
    assert _v(mx, M=0, x=None, y=None) == 0 and _v(mx, N=0, codes=None, y=None) == 0
    assert _v(mx, y=None) == -1 and _v(mx, ldy=32) == -1
    assert _v(mx, codes=None) == -1 and _v(mx, scales=None) == -1 and _v(mx, x=None) == -1 and _v(mx, ldx=128) == -1
    assert _v(mx, y=17) == -2 and _v(mx, y=18, ydt=0) == -2
    assert _v(mx, codes=8) == -2 and _v(mx, scales=8) == -2 and _v(mx, x=8) == -2 and _v(mx, ldx=260) == -2
    assert _v(mx, M=65537) == -4 and _v(mx, N=1 << 31, ldy=1 << 31) == -4
    assert _v(mx, N=1 << 20, ldy=1 << 20, K=1 << 17, ldx=1 << 17) == -4   # 4 GiB of scales


def test_gemv_nvfp4_refusals(mx):
    L = mx.lib()

    def call(codes=16, scales=16, enc=16, dom=0, sl=1, x=16, ldx=256, M=1, N=64, K=256, y=16, ldy=64):
        return L.mx_gemv_nvfp4(codes, scales, enc, dom, sl, x, 1, ldx, M, N, K, 1.0, y, 1, ldy, None)

    assert call(K=24) == -3 and call(dom=-1) == -1 and call(enc=None) == -1 and call(enc=18) == -2
    assert call(sl=3) == -1 and call(scales=8) == -2 and call(M=0, enc=None) == 0


def test_packed_refusals(mx):
    """A record goes through the same checks; fields out of their types' range are refused."""
    L = mx.lib()
    norm = [16, 1, 4, 64, 64, 0, 0, 16, 1, 1e-5, 0, 0, 0, 0, 0, 0, 16, 64, 0, 0, 0, 0, 0]
    back = [16, 1, 4, 64, 64, 16, 64, 16, 1, 16, 0, 0, 16, 64, 16, 16, 4 * 64 * 4, 0]
    gemv = [16, 16, 0, 4, 0, 0, 1, 16, 1, 256, 1, 64, 256, 1.0, 16, 1, 64, 0]

    def call(name, record, pack, **change):
        r = list(record)
        for k, v in change.items():
            r[int(k[1:])] = v
        return getattr(L, name)(pack(*r))

    n = lambda **c: call("mx_rmsnorm_packed", norm, mx._NORM_RECORD, **c)            # noqa: E731
    b = lambda **c: call("mx_rmsnorm_backward_packed", back, mx._BACKWARD_RECORD, **c)   # noqa: E731
    v = lambda **c: call("mx_gemv_packed", gemv, mx._GEMV_RECORD, **c)               # noqa: E731
    assert L.mx_rmsnorm_packed(None) == L.mx_rmsnorm_backward_packed(None) == L.mx_gemv_packed(None) == -1
    assert n(_0=0) == -1 and n(_1=2 ** 32 + 1) == -1 and n(_3=48) == -3 and n(_0=8) == -2 and n(_2=0) == 0
    assert n(_10=1) == -1 and n(_10=1, _19=16, _20=16, _21=2 ** 32) == -1 and n(_10=1, _19=24, _20=16, _21=1) == -2
    assert n(_10=1, _19=16, _20=16, _11=-1) == -1 and n(_16=0) == -1 and n(_14=16) == -1 and n(_9=1e300) == -1
    assert b(_0=0) == -1 and b(_16=4 * 64 * 4 - 1) == -1 and b(_16=-1) == -1 and b(_14=2) == -2 and b(_3=48) == -3
    assert b(_3=0, _0=0) == 0 and b(_8=2 ** 32) == -1
    assert v(_3=0) == -4 and v(_3=2 ** 33 + 4) == -1 and v(_12=48) == -3 and v(_0=8) == -2 and v(_10=0) == 0
    assert v(_2=1) == -1 and v(_2=1, _4=18) == -2 and v(_2=1, _4=16, _12=24) == -3 and v(_15=2) == -1


def test_binding_refuses_before_the_library(mx):
    """Tensors that are not on the GPU, or of another shape or type, never reach a kernel."""
    x, w = torch.zeros(4, 64), torch.zeros(64)
    u8 = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mx.rmsnorm(x, w)
    with pytest.raises(ValueError):
        mx.rmsnorm(x.t(), w)
    with pytest.raises(TypeError):
        mx.rmsnorm(x.double(), w)
    with pytest.raises(ValueError):
        mx.rmsnorm_quantize(x, w)
    with pytest.raises(ValueError):
        mx.rmsnorm_backward(x, x, w, torch.zeros(4))
    with pytest.raises(ValueError):
        mx.gemv(u8, u8, x, 16, 64)
    with pytest.raises(ValueError):
        mx.gemv(u8, u8, x, 16, 32)                 # x has another K
    with pytest.raises(ValueError):
        mx.gemv_nvfp4((u8, u8, torch.zeros(1)), x, 16, 64)


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu(mx):
    d = dict(device="cuda")
    x, w = torch.zeros(4, 64, **d), torch.zeros(64, **d)
    u8 = torch.zeros(4096, dtype=torch.uint8, **d)
    with pytest.raises(ValueError):
        mx.rmsnorm(x, w.cpu())
    with pytest.raises(ValueError):
        mx.rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        mx.rmsnorm(x, w, residual=x[:3])
    with pytest.raises(TypeError):
        mx.rmsnorm(x, w, residual=x.bfloat16())
    with pytest.raises(ValueError):
        mx.rmsnorm(x, w, out=(None, torch.empty_like(x), None))
    with pytest.raises(ValueError):
        mx.rmsnorm_quantize(x, w, out=(u8[:255], None, None, None, None))
    with pytest.raises(ValueError):
        mx.rmsnorm_quantize(x, w, out=(None, u8[:511], None, None, None))
    with pytest.raises(ValueError):
        mx.rmsnorm_backward(x, x, w, torch.zeros(3, **d))
    with pytest.raises(ValueError):
        mx.rmsnorm_backward(x, x, w, torch.zeros(4, **d), workspace=u8[:1023])
    with pytest.raises(ValueError):
        mx.gemv(u8[:511], u8, x, 16, 64)
    with pytest.raises(ValueError):
        mx.gemv(u8, u8[:511], x, 16, 64)
    with pytest.raises(ValueError):
        mx.gemv(u8, u8, x, 16, 64, out=torch.empty(4, 17, **d))
    with pytest.raises(ValueError):
        mx.gemv_nvfp4((u8, u8, torch.zeros(1, **d)), x, 16, 64, domain_rows=8)
    with pytest.raises(mx.MxError):
        mx.rmsnorm(torch.zeros(4, 66, **d)[:, 2:], w)     # rows not 16-byte aligned
    torch.cuda.synchronize()
