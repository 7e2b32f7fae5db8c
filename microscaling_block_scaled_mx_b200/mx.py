"""Thin Python binding of libmx (include/mx.h): argument marshalling only.

Every step of the cast and of the GEMM runs in the CUDA kernels of libmx.so;
PyTorch only provides device memory and streams.  There is no CPU fallback:
if libmx.so is missing or fails to load, every call raises.

Functions take and return torch tensors on the current CUDA device; bf16 and
fp32 inputs are accepted, codes and scales are uint8 tensors laid out as
documented in include/mx.h.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmx.so")

FMT = {"e4m3": 0, "e5m2": 1, "e2m3": 2, "e3m2": 3, "e2m1": 4, "int8": 5}
FMT_BITS = {0: 8, 1: 8, 2: 6, 3: 6, 4: 4, 5: 8}
ROUND = {"rne": 0, "sr": 1}
LAYOUT = {"plain": 0, "mma": 1, "mma_x4": 2}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
DEFAULT_SIGN_MASK = 0x6A09E667

MX_OK = 0
STATUS_NAMES = {0: "MX_OK", -1: "MX_ERR_ARG", -2: "MX_ERR_ALIGN", -3: "MX_ERR_SHAPE",
                -4: "MX_ERR_UNSUPPORTED", -5: "MX_ERR_SR_RANGE", -6: "MX_ERR_CUDA",
                -7: "MX_ERR_TIMEOUT", -8: "MX_ERR_BOUNDS"}


class MxError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} ({status})")


class _Precond(ctypes.Structure):
    _fields_ = [("hadamard", ctypes.c_int32), ("sign_mask", ctypes.c_uint32)]


class _Shard(ctypes.Structure):
    _fields_ = [("row0", ctypes.c_int64), ("col0", ctypes.c_int64),
                ("total_rows", ctypes.c_int64), ("total_cols", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load libmx.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libmx.so not found at {LIB_PATH}; build it with "
                    "`python -m microscaling_block_scaled_mx_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, i32, u32, u64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                      ctypes.c_uint32, ctypes.c_uint64)
            L.mx_quantize.restype = i32
            L.mx_quantize.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, u64,
                                      ctypes.POINTER(_Precond), vp, vp, i32, vp]
            L.mx_quantize_shard.restype = i32
            L.mx_quantize_shard.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, u64,
                                            ctypes.POINTER(_Precond), ctypes.POINTER(_Shard), vp, vp, i32, vp]
            L.mx_quantize_dual_shard.restype = i32
            L.mx_quantize_dual_shard.argtypes = [vp, i32, i64, i64, i64, i32, i32, u64, i32, u64,
                                                 ctypes.POINTER(_Precond), ctypes.POINTER(_Shard),
                                                 vp, vp, vp, vp, i32, vp]
            L.mx_quantize_dual.restype = i32
            L.mx_quantize_dual.argtypes = [vp, i32, i64, i64, i64, i32, i32, u64, i32, u64,
                                           ctypes.POINTER(_Precond), vp, vp, vp, vp, i32, vp]
            L.mx_quantize_nvfp4.restype = i32
            L.mx_quantize_nvfp4.argtypes = [vp, i32, i64, i64, i64, i64, vp, vp, i32, vp, vp]
            L.mx_nvfp4_scales_bytes.restype = ctypes.c_size_t
            L.mx_nvfp4_scales_bytes.argtypes = [i32, i64, i64]
            L.mx_nvfp4_domains.restype = i64
            L.mx_nvfp4_domains.argtypes = [i64, i64]
            L.mx_dequantize.restype = i32
            L.mx_dequantize.argtypes = [vp, vp, i32, i32, i64, i64, vp, i32, i64, vp]
            L.mx_gemm.restype = i32
            L.mx_gemm.argtypes = [vp, vp, i32, vp, vp, i32, i64, i64, i64, ctypes.c_float,
                                  vp, i32, i64, vp, ctypes.c_size_t, vp]
            L.mx_gemm_nvfp4_x4.restype = i32
            L.mx_gemm_nvfp4_x4.argtypes = [vp, vp, vp, i64, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float,
                                           vp, i32, i64, vp]
            L.mx_gemm_nvfp4.restype = i32
            L.mx_gemm_nvfp4.argtypes = [vp, vp, vp, i64, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float,
                                        vp, i32, i64, vp]
            L.mx_gemm_x4.restype = i32
            L.mx_gemm_x4.argtypes = [vp, vp, i32, vp, vp, i32, i64, i64, i64, ctypes.c_float, vp, i32, i64, vp]
            L.mx_gemm_quantize_x4.restype = i32
            L.mx_gemm_quantize_x4.argtypes = [vp, vp, i32, vp, vp, i32, i64, i64, i64, ctypes.c_float,
                                              i32, i32, u64, vp, vp, i32, vp]
            L.mx_gemm_quantize.restype = i32
            L.mx_gemm_quantize.argtypes = [vp, vp, i32, vp, vp, i32, i64, i64, i64, ctypes.c_float,
                                           i32, i32, u64, vp, vp, i32, vp]
            for name in ("mx_rmsnorm_packed", "mx_rmsnorm_backward_packed", "mx_gemv_packed"):
                getattr(L, name).restype = i32
                getattr(L, name).argtypes = [ctypes.c_char_p]
            L.mx_rmsnorm_backward_workspace_bytes.restype = ctypes.c_size_t
            L.mx_rmsnorm_backward_workspace_bytes.argtypes = [i64, i64]
            L.mx_codes_bytes.restype = ctypes.c_size_t
            L.mx_codes_bytes.argtypes = [i32, i64, i64]
            L.mx_scales_bytes.restype = ctypes.c_size_t
            L.mx_scales_bytes.argtypes = [i32, i64, i64]
            L.mx_gemm_workspace_bytes.restype = ctypes.c_size_t
            L.mx_gemm_workspace_bytes.argtypes = [i64, i64, i64]
            L.mx_last_device_status.restype = i32
            L.mx_last_device_status.argtypes = [vp]
            L.mx_status_str.restype = ctypes.c_char_p
            L.mx_status_str.argtypes = [i32]
            L.mx_abi_version.restype = i32
            L.mx_abi_version.argtypes = []
            L.mx_debug_gemm_skip_stage.restype = i32
            L.mx_debug_gemm_skip_stage.argtypes = [i32]
            L.mx_debug_gemm_force_kernel.restype = i32
            L.mx_debug_gemm_force_kernel.argtypes = [i32]
            L.mx_debug_cast_force_cpasync.restype = i32
            L.mx_debug_cast_force_cpasync.argtypes = [i32]
            L.mx_debug_cast_skip_tile.restype = i32
            L.mx_debug_cast_skip_tile.argtypes = [i32]
            L.mx_debug_cast_cut_codes_cap.restype = i32
            L.mx_debug_cast_cut_codes_cap.argtypes = [i64]
            _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().mx_status_str(status).decode()


def _fmt(f) -> int:
    return FMT[f] if isinstance(f, str) else int(f)


def _layout(sl) -> int:
    return LAYOUT[sl] if isinstance(sl, str) else int(sl)


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(rc: int, what: str) -> None:
    if rc != MX_OK:
        raise MxError(rc, what)


def codes_bytes(fmt, outer: int, inner: int) -> int:
    return lib().mx_codes_bytes(_fmt(fmt), outer, inner)


def scales_bytes(scale_layout, outer: int, inner: int) -> int:
    return lib().mx_scales_bytes(_layout(scale_layout), outer, inner)


def codes_row_bytes(fmt, inner: int) -> int:
    return inner * FMT_BITS[_fmt(fmt)] // 8


def quantize(x: torch.Tensor, block_axis: int = 1, fmt="e4m3", rnd="rne", seed: int = 0,
             hadamard: bool = False, sign_mask: int = DEFAULT_SIGN_MASK, scale_layout="mma",
             codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
             stream=None, shard=None):
    """MX cast of a 2-D CUDA tensor (rows x cols, row pitch x.stride(0)).

    Returns (codes, scales): codes is (outer, packed_inner_bytes) uint8 with
    outer = rows for block_axis=1 and cols for block_axis=0; scales is flat.
    shard = (row0, col0, total_rows, total_cols) casts x as the piece at
    (row0, col0) of a larger tensor (mx_quantize_shard).
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype not in DTYPE:
        raise TypeError("x must be float32 or bfloat16")
    f = _fmt(fmt)
    sl = _layout(scale_layout)
    rows, cols = x.shape
    outer, inner = (rows, cols) if block_axis == 1 else (cols, rows)
    if codes is None:
        codes = torch.empty((outer, codes_row_bytes(f, inner)), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(max(scales_bytes(sl, outer, inner), 1), dtype=torch.uint8, device=x.device)
    pre = _Precond(1 if hadamard else 0, sign_mask & 0xFFFFFFFF)
    r = ROUND[rnd] if isinstance(rnd, str) else int(rnd)
    if shard is None:
        rc = lib().mx_quantize(x.data_ptr(), DTYPE[x.dtype], rows, cols, x.stride(0), block_axis, f,
                               r, seed & (2**64 - 1), ctypes.byref(pre), codes.data_ptr(), scales.data_ptr(),
                               sl, _stream(stream))
        _check(rc, "mx_quantize")
    else:
        sh = _Shard(*shard)
        rc = lib().mx_quantize_shard(x.data_ptr(), DTYPE[x.dtype], rows, cols, x.stride(0), block_axis, f,
                                     r, seed & (2**64 - 1), ctypes.byref(pre), ctypes.byref(sh),
                                     codes.data_ptr(), scales.data_ptr(), sl, _stream(stream))
        _check(rc, "mx_quantize_shard")
    return codes, scales


def quantize_dual(x: torch.Tensor, fmt="e4m3", rnd_rows="rne", seed_rows: int = 0, rnd_cols="rne",
                  seed_cols: int = 0, hadamard: bool = False, sign_mask: int = DEFAULT_SIGN_MASK,
                  scale_layout="mma", out=None, stream=None, shard=None):
    """Both MX casts of a 2-D CUDA tensor from one read of it.

    Returns (codes_rows, scales_rows, codes_cols, scales_cols): the results of
    quantize(x, 1, ...) with (rnd_rows, seed_rows) and of quantize(x, 0, ...)
    with (rnd_cols, seed_cols, hadamard); `out` may supply the four buffers.
    shard = (row0, col0, total_rows, total_cols) casts x as that piece of a
    larger tensor (mx_quantize_dual_shard).
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype not in DTYPE:
        raise TypeError("x must be float32 or bfloat16")
    f = _fmt(fmt)
    sl = _layout(scale_layout)
    rows, cols = x.shape
    if out is None:
        u8 = dict(dtype=torch.uint8, device=x.device)
        out = (torch.empty((rows, codes_row_bytes(f, cols)), **u8),
               torch.empty(max(scales_bytes(sl, rows, cols), 1), **u8),
               torch.empty((cols, codes_row_bytes(f, rows)), **u8),
               torch.empty(max(scales_bytes(sl, cols, rows), 1), **u8))
    cr, sr_, cc, sc = out
    pre = _Precond(1 if hadamard else 0, sign_mask & 0xFFFFFFFF)
    rnd = lambda r: ROUND[r] if isinstance(r, str) else int(r)
    if shard is None:
        rc = lib().mx_quantize_dual(x.data_ptr(), DTYPE[x.dtype], rows, cols, x.stride(0), f,
                                    rnd(rnd_rows), seed_rows & (2**64 - 1), rnd(rnd_cols), seed_cols & (2**64 - 1),
                                    ctypes.byref(pre), cr.data_ptr(), sr_.data_ptr(), cc.data_ptr(), sc.data_ptr(),
                                    sl, _stream(stream))
        _check(rc, "mx_quantize_dual")
    else:
        sh = _Shard(*shard)
        rc = lib().mx_quantize_dual_shard(x.data_ptr(), DTYPE[x.dtype], rows, cols, x.stride(0), f,
                                          rnd(rnd_rows), seed_rows & (2**64 - 1), rnd(rnd_cols),
                                          seed_cols & (2**64 - 1), ctypes.byref(pre), ctypes.byref(sh),
                                          cr.data_ptr(), sr_.data_ptr(), cc.data_ptr(), sc.data_ptr(),
                                          sl, _stream(stream))
        _check(rc, "mx_quantize_dual_shard")
    return cr, sr_, cc, sc


def quantize_nvfp4(x: torch.Tensor, domain_rows: int = 0, scale_layout="mma", out=None, stream=None):
    """NVFP4 cast of a 2-D CUDA tensor along its rows (mx_quantize_nvfp4):
    domain_rows 0 for one global scale domain, else rows per CTA-local domain.
    Returns (codes, scales, enc_scales)."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype not in DTYPE:
        raise TypeError("x must be float32 or bfloat16")
    rows, cols = x.shape
    sl = _layout(scale_layout)
    if out is None:
        u8 = dict(dtype=torch.uint8, device=x.device)
        out = (torch.empty((rows, cols // 2), **u8),
               torch.empty(max(lib().mx_nvfp4_scales_bytes(sl, rows, cols), 1), **u8),
               torch.empty(max(lib().mx_nvfp4_domains(rows, domain_rows), 1), dtype=torch.float32,
                           device=x.device))
    codes, scales, enc = out
    rc = lib().mx_quantize_nvfp4(x.data_ptr(), DTYPE[x.dtype], rows, cols, x.stride(0), domain_rows,
                                 codes.data_ptr(), scales.data_ptr(), sl, enc.data_ptr(), _stream(stream))
    _check(rc, "mx_quantize_nvfp4")
    return codes, scales, enc


def dequantize(codes: torch.Tensor, scales: torch.Tensor, fmt, outer: int, inner: int,
               scale_layout="mma", out_dtype=torch.float32, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Exact decode X * P, rounded once to out_dtype; returns (outer, inner)."""
    if out is None:
        out = torch.empty((outer, inner), dtype=out_dtype, device=codes.device)
    rc = lib().mx_dequantize(codes.data_ptr(), scales.data_ptr(), _fmt(fmt), _layout(scale_layout),
                             outer, inner, out.data_ptr(), DTYPE[out.dtype], out.stride(0),
                             _stream(stream))
    _check(rc, "mx_dequantize")
    return out


def gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
         b_scales: torch.Tensor, M: int, N: int, K: int, fa="e4m3", fb=None, alpha: float = 1.0,
         out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None,
         scale_layout="mma") -> torch.Tensor:
    """C = alpha * A * B^T on MX operands quantized along K; scale_layout is the
    operands' scale layout, "mma" (mx_gemm) or "mma_x4" (mx_gemm_x4)."""
    fb = fa if fb is None else fb
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    args = (a_codes.data_ptr(), a_scales.data_ptr(), _fmt(fa), b_codes.data_ptr(), b_scales.data_ptr(), _fmt(fb),
            M, N, K, float(alpha), out.data_ptr(), DTYPE[out.dtype], out.stride(0))
    if _layout(scale_layout) == LAYOUT["mma_x4"]:
        rc = lib().mx_gemm_x4(*args, _stream(stream))
        _check(rc, "mx_gemm_x4")
    elif _layout(scale_layout) == LAYOUT["mma"]:
        rc = lib().mx_gemm(*args, None, 0, _stream(stream))
        _check(rc, "mx_gemm")
    else:
        raise ValueError("GEMM operand scales are in the mma or mma_x4 layout")
    return out


def gemm_nvfp4(a, b, M: int, N: int, K: int, a_domain_rows: int = 0, b_domain_rows: int = 0,
               alpha: float = 1.0, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
               stream=None, scale_layout="mma") -> torch.Tensor:
    """C = alpha * A * B^T on NVFP4 operands (mx_gemm_nvfp4, or mx_gemm_nvfp4_x4
    for scale_layout "mma_x4"): a and b are the (codes, scales, enc_scales)
    triples quantize_nvfp4 returns in that layout."""
    (ac, asc, ae), (bc, bsc, be) = a, b
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=ac.device)
    fn = {LAYOUT["mma"]: "mx_gemm_nvfp4", LAYOUT["mma_x4"]: "mx_gemm_nvfp4_x4"}.get(_layout(scale_layout))
    if fn is None:
        raise ValueError("NVFP4 GEMM operand scales are in the mma or mma_x4 layout")
    rc = getattr(lib(), fn)(ac.data_ptr(), asc.data_ptr(), ae.data_ptr(), a_domain_rows,
                            bc.data_ptr(), bsc.data_ptr(), be.data_ptr(), b_domain_rows, M, N, K,
                            float(alpha), out.data_ptr(), DTYPE[out.dtype], out.stride(0), _stream(stream))
    _check(rc, fn)
    return out


def gemm_quantize(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
                  b_scales: torch.Tensor, M: int, N: int, K: int, fa="e4m3", fb=None, alpha: float = 1.0,
                  out_fmt="e4m3", rnd="rne", seed: int = 0, scale_layout="mma", out=None, stream=None,
                  operand_layout="mma"):
    """alpha * A * B^T quantized along its rows in the GEMM epilogue.

    Returns (codes, scales): M x (N * bits / 8) codes and the scales of an
    M x N tensor in `scale_layout`; `out` may supply both buffers."""
    fb = fa if fb is None else fb
    of = _fmt(out_fmt)
    sl = _layout(scale_layout)
    if out is None:
        dev = a_codes.device
        out = (torch.empty((M, codes_row_bytes(of, N)), dtype=torch.uint8, device=dev),
               torch.empty(max(scales_bytes(sl, M, N), 1), dtype=torch.uint8, device=dev))
    codes, scales = out
    fn = {LAYOUT["mma"]: "mx_gemm_quantize", LAYOUT["mma_x4"]: "mx_gemm_quantize_x4"}.get(_layout(operand_layout))
    if fn is None:
        raise ValueError("GEMM operand scales are in the mma or mma_x4 layout")
    rc = getattr(lib(), fn)(a_codes.data_ptr(), a_scales.data_ptr(), _fmt(fa), b_codes.data_ptr(),
                            b_scales.data_ptr(), _fmt(fb), M, N, K, float(alpha), of,
                            ROUND[rnd] if isinstance(rnd, str) else int(rnd), seed & (2**64 - 1),
                            codes.data_ptr(), scales.data_ptr(), sl, _stream(stream))
    _check(rc, fn)
    return codes, scales


# The checks of the calls below.  They read each tensor attribute once: a
# decoding step makes these calls for every layer and token, and on tensors of
# a few kilobytes the host's part is most of their time.

# The records of mx_rmsnorm_packed, mx_rmsnorm_backward_packed and mx_gemv_packed
# (include/mx.h): addresses, numbers and two doubles, eight bytes each.
_NORM_RECORD = struct.Struct("=Q4qQqQqd3qQQqQqQQQqQ").pack
_BACKWARD_RECORD = struct.Struct("=Q4qQqQqQQqQqQQqQ").pack
_GEMV_RECORD = struct.Struct("=QQqqQqqQ5qdQqqQ").pack

# torch's helpers behind torch.cuda.current_device and current_stream, which make
# no wrapper objects; a torch without them (a CPU build) has the public functions.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _device(t: torch.Tensor, what: str) -> int:
    """The index of t's device, which has to be the current one."""
    device = t.get_device()
    if device < 0 or device != _current_device():
        raise ValueError(f"{what} must be on the current CUDA device")
    return device


def _elsewhere(what: str):
    raise ValueError(f"{what} must be on the same CUDA device as the other tensors")


def _first(t: torch.Tensor, what: str):
    """Check the 2-D tensor that gives a call its device, type and sizes;
    returns (device, dtype code, shape, leading dimension)."""
    dt = DTYPE.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what} must be float32 or bfloat16")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what} must be 2-D with unit column stride")
    return _device(t, what), dt, shape, strides[0] if shape[0] > 1 else shape[1]


def _matrix(device: int, t: torch.Tensor, what: str, shape, dtype) -> int:
    """Check a 2-D row-pitched tensor; returns its leading dimension."""
    if t.get_device() != device:
        _elsewhere(what)
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    strides = t.stride()
    if t.shape != shape or (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what} must be {shape[0]} x {shape[1]} with unit column stride")
    return strides[0] if shape[0] > 1 else shape[1]


def _flat(device: int, t: torch.Tensor, what: str, n: int, dtype) -> int:
    """Check a contiguous buffer of at least n values; returns its address."""
    if t.get_device() != device:
        _elsewhere(what)
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous and hold {n} values")
    return t.data_ptr()


def _weight(device: int, t: torch.Tensor, cols: int):
    """Check a norm's weight; returns (address, dtype code)."""
    if t.get_device() != device:
        _elsewhere("weight")
    dt = DTYPE.get(t.dtype)
    if dt is None:
        raise TypeError("weight must be float32 or bfloat16")
    if t.numel() != cols or not t.is_contiguous():
        raise ValueError(f"weight must be contiguous and hold {cols} values")
    return t.data_ptr(), dt


def _empty(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """A new contiguous tensor on like's device, which belongs to the stream that
    the call runs on.  (torch.empty takes 1 us longer than empty_strided.)"""
    strides = (shape[1], 1) if len(shape) == 2 else (1,)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)


def _scale_bytes(layout: int, outer: int, blocks: int) -> int:
    """mx_scales_bytes of `blocks` scales per row, without a call into the library."""
    if layout == 0:
        return outer * blocks
    if layout not in (1, 2):
        return 0                        # refused by the call
    return -(-outer // 128) * 128 * (-(-blocks // 4) * 4) * (4 if layout == 2 else 1)


def _handle(stream, device: int) -> int:
    """The stream's handle; of the current stream without a Stream object."""
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _norm_args(x, weight, residual, h, y, want_y, rstd, want_rstd, stream):
    """Checks and allocations that the norm's two forms share."""
    dev, xdt, shape, ldx = _first(x, "x")
    rows, cols = shape
    w, wdt = _weight(dev, weight, cols)
    if residual is not None and h is None:
        h = _empty(shape, x.dtype, x, stream)
    if want_y and y is None:
        y = _empty(shape, x.dtype, x, stream)
    if want_rstd and rstd is None:
        rstd = _empty((rows,), torch.float32, x, stream)
    r = hp = yp = rp = ldr = ldh = ldy = 0
    if residual is not None:
        ldr = _matrix(dev, residual, "residual", shape, x.dtype)
        ldh = _matrix(dev, h, "h", shape, x.dtype)
        r, hp = residual.data_ptr(), h.data_ptr()
    elif h is not None:
        raise ValueError("h is written only with a residual")
    if y is not None:
        ldy = _matrix(dev, y, "y", shape, x.dtype)
        yp = y.data_ptr()
    if rstd is not None:
        rp = _flat(dev, rstd, "rstd", rows, torch.float32)
    return (x.data_ptr(), xdt, rows, cols, ldx, r, ldr, w, wdt), (hp, ldh, yp, ldy, rp), dev, h, y, rstd


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: torch.Tensor | None = None,
            with_rstd: bool = False, out=None, stream=None):
    """RMS norm of each row of a 2-D CUDA tensor (mx_rmsnorm), after adding
    `residual` to it if one is given.

    Returns (y, h, rstd): y in x's type, h = x + residual (None without a
    residual), rstd the rows' 1 / sqrt(mean square + eps) as fp32 (None unless
    asked for).  `out` may supply the three; h may be x or the residual itself
    and y may be x."""
    y, h, rstd = out if out is not None else (None, None, None)
    ins, outs, dev, h, y, rstd = _norm_args(x, weight, residual, h, y, True, rstd, with_rstd, stream)
    rc = (_lib or lib()).mx_rmsnorm_packed(_NORM_RECORD(*ins, eps, 0, 0, 0, 0, *outs, 0, 0, 0, _handle(stream, dev)))
    if rc != MX_OK:
        raise MxError(rc, "mx_rmsnorm")
    return y, h, rstd


def rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
                     residual: torch.Tensor | None = None, fmt="e4m3", rnd="rne", seed: int = 0,
                     scale_layout="mma", with_y: bool = False, with_rstd: bool = False, out=None, stream=None):
    """The RMS norm of rmsnorm, cast along its rows (mx_rmsnorm_quantize).

    Returns (codes, scales, h, y, rstd): the codes and scales of
    quantize(y, 1, fmt, ...) on the fp32 y; h, y and rstd as in rmsnorm, each
    None unless there is a residual, with_y, with_rstd.  `out` may supply the
    five (None for one that is not wanted or is to be allocated)."""
    codes, scales, h, y, rstd = out if out is not None else (None,) * 5
    ins, outs, dev, h, y, rstd = _norm_args(x, weight, residual, h, y, with_y, rstd, with_rstd, stream)
    f, sl = _fmt(fmt), _layout(scale_layout)
    L = _lib or lib()
    rows, cols = ins[2], ins[3]
    row_bytes = cols * FMT_BITS.get(f, 0) // 8
    n_scales = _scale_bytes(sl, rows, -(-cols // 32))
    if codes is None:
        codes = _empty((rows, row_bytes), torch.uint8, x, stream)
    if scales is None:
        scales = _empty((max(n_scales, 1),), torch.uint8, x, stream)
    c = _flat(dev, codes, "codes", rows * row_bytes, torch.uint8)
    s = _flat(dev, scales, "scales", n_scales, torch.uint8)
    rc = L.mx_rmsnorm_packed(_NORM_RECORD(*ins, eps, 1, f, ROUND[rnd] if isinstance(rnd, str) else int(rnd),
                                          seed & (2**64 - 1), *outs, c, s, sl, _handle(stream, dev)))
    if rc != MX_OK:
        raise MxError(rc, "mx_rmsnorm_quantize")
    return codes, scales, h, y, rstd


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dres: torch.Tensor | None = None, out=None, workspace: torch.Tensor | None = None,
                     stream=None):
    """Gradients of rmsnorm (mx_rmsnorm_backward): h and rstd as the forward
    pass returned them (h = x without a residual), dres the gradient that
    reaches h by its other uses.

    Returns (dx, dweight): dx in dy's type, the gradient of x and of the
    residual, and dweight as fp32.  `out` may supply both (dx may be dy or
    dres), `workspace` the uint8 scratch of rmsnorm_backward_workspace, which
    one call at a time may use."""
    dev, dt, shape, lddy = _first(dy, "dy")
    rows, cols = shape
    dx, dweight = out if out is not None else (None, None)
    L = _lib or lib()
    n_ws = min(rows, 296) * cols * 4             # mx_rmsnorm_backward_workspace_bytes
    if dx is None:
        dx = _empty(shape, dy.dtype, dy, stream)
    if dweight is None:
        dweight = _empty((cols,), torch.float32, dy, stream)
    if workspace is None:
        workspace = _empty((max(n_ws, 1),), torch.uint8, dy, stream)
    ldh = _matrix(dev, h, "h", shape, dy.dtype)
    lddx = _matrix(dev, dx, "dx", shape, dy.dtype)
    lddres = _matrix(dev, dres, "dres", shape, dy.dtype) if dres is not None else 0
    w, wdt = _weight(dev, weight, cols)
    rp = _flat(dev, rstd, "rstd", rows, torch.float32)
    dwp = _flat(dev, dweight, "dweight", cols, torch.float32)
    wsp = _flat(dev, workspace, "workspace", n_ws, torch.uint8)
    rc = L.mx_rmsnorm_backward_packed(_BACKWARD_RECORD(
        dy.data_ptr(), dt, rows, cols, lddy, h.data_ptr(), ldh, w, wdt, rp, 0 if dres is None else dres.data_ptr(), lddres,
        dx.data_ptr(), lddx, dwp, wsp, workspace.numel(), _handle(stream, dev)))
    if rc != MX_OK:
        raise MxError(rc, "mx_rmsnorm_backward")
    return dx, dweight


def rmsnorm_backward_workspace(rows: int, cols: int, device=None) -> torch.Tensor:
    """Scratch for rmsnorm_backward on rows x cols."""
    n = lib().mx_rmsnorm_backward_workspace_bytes(rows, cols)
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda" if device is None else device)


def _gemv_args(x, N, K, out_dtype, out, stream):
    """Checks and allocations that the two weight formats share."""
    dev, xdt, shape, ldx = _first(x, "x")
    if shape[1] != K:
        raise ValueError("x must have K columns")
    M = shape[0]
    if out is None:
        out = _empty((M, N), x.dtype if out_dtype is None else out_dtype, x, stream)
    ydt = DTYPE.get(out.dtype)
    if ydt is None:
        raise TypeError("the output must be float32 or bfloat16")
    ldy = _matrix(dev, out, "out", (M, N), out.dtype)
    return dev, out, (x.data_ptr(), xdt, ldx, M, N, K), (out.data_ptr(), ydt, ldy)


def gemv(w_codes: torch.Tensor, w_scales: torch.Tensor, x: torch.Tensor, N: int, K: int, fmt="e2m1",
         alpha: float = 1.0, out_dtype=None, out: torch.Tensor | None = None, scale_layout="mma",
         stream=None) -> torch.Tensor:
    """y = alpha * x W^T for the few tokens of x (M x K, not quantized) and N x K
    MXFP4 weights (mx_gemv): the (codes, scales) quantize returns for W along K
    in `scale_layout`, the buffers gemm takes as its B operand.  The output has
    x's type unless out_dtype or `out` says otherwise."""
    f, sl = _fmt(fmt), _layout(scale_layout)
    dev, out, ins, outs = _gemv_args(x, N, K, out_dtype, out, stream)
    L = _lib or lib()
    c = _flat(dev, w_codes, "w_codes", N * K // 2, torch.uint8)
    s = _flat(dev, w_scales, "w_scales", _scale_bytes(sl, N, -(-K // 32)), torch.uint8)
    rc = L.mx_gemv_packed(_GEMV_RECORD(c, s, 0, f, 0, 0, sl, *ins, alpha, *outs, _handle(stream, dev)))
    if rc != MX_OK:
        raise MxError(rc, "mx_gemv")
    return out


def gemv_nvfp4(w, x: torch.Tensor, N: int, K: int, domain_rows: int = 0, alpha: float = 1.0, out_dtype=None,
               out: torch.Tensor | None = None, scale_layout="mma", stream=None) -> torch.Tensor:
    """gemv with NVFP4 weights (mx_gemv_nvfp4): w is the (codes, scales,
    enc_scales) triple quantize_nvfp4 returns for W with `domain_rows` in
    `scale_layout`."""
    codes, scales, enc = w
    sl = _layout(scale_layout)
    dev, out, ins, outs = _gemv_args(x, N, K, out_dtype, out, stream)
    L = _lib or lib()
    c = _flat(dev, codes, "codes", N * K // 2, torch.uint8)
    s = _flat(dev, scales, "scales", _scale_bytes(sl, N, -(-K // 16)), torch.uint8)
    domains = -(-N // domain_rows) if domain_rows > 0 else 1         # a negative one is refused by the call
    e = _flat(dev, enc, "enc_scales", domains, torch.float32)
    rc = L.mx_gemv_packed(_GEMV_RECORD(c, s, 1, 0, e, domain_rows, sl, *ins, alpha, *outs, _handle(stream, dev)))
    if rc != MX_OK:
        raise MxError(rc, "mx_gemv_nvfp4")
    return out


def last_device_status(stream=None) -> int:
    return lib().mx_last_device_status(_stream(stream))
