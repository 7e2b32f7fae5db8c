"""The RMS norms that end in an MX cast and the products of a few tokens with
4-bit weights, as a program calls them, with their plain forms and their
definition in 64 bits.

Operators
  norm           h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight
  norm_cast      the same, y as MX codes and scales along its rows
  norm_backward  gradients of the norm with respect to h and the weight
  gemv           y = x W^T, W in MXFP4 (E2M1 codes, an E8M0 scale per 32)
  gemv_nvfp4     y = x W^T, W in NVFP4 (E2M1 codes, an E4M3 scale per 16, fp32
                 encode scales per domain of rows)
"""
import math

import torch

own = False

EPS = 1e-5
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
EMAX = {"e4m3": 8, "e5m2": 15, "e2m1": 2}
MAXV = {"e4m3": 448.0, "e5m2": 57344.0}
MANT = {"e4m3": 3, "e5m2": 2}
EMIN = {"e4m3": -6, "e5m2": -14}
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one token of a decoder, hidden size 4096: the norm in front of a 4-bit projection
        dict(name="norm_decode_1x4096", op="norm", rows=1, cols=4096, dtype="bf16", residual=True),
        # a decoding batch whose projections run as block-scaled products
        dict(name="norm_cast_64x4096", op="norm_cast", rows=64, cols=4096, dtype="bf16", residual=True, fmt="e4m3",
             layout="mma", train=False),
        # odd row and block counts, fp32, no residual: the first norm of a small model; y and 1/rms kept for training
        dict(name="norm_cast_1013x1056_f32", op="norm_cast", rows=1013, cols=1056, dtype="fp32", residual=False,
             fmt="e5m2", layout="plain", train=True),
        # a training step's (or a long prompt's) tokens
        dict(name="norm_cast_16384x4096", op="norm_cast", rows=16384, cols=4096, dtype="bf16", residual=True,
             fmt="e4m3", layout="mma_x4", train=False),
        # the backward pass over 8192 tokens, with the gradient of the residual stream
        dict(name="norm_backward_8192x4096", op="norm_backward", rows=8192, cols=4096, dtype="bf16", residual=True),
        # a short, odd batch in fp32
        dict(name="norm_backward_333x1056_f32", op="norm_backward", rows=333, cols=1056, dtype="fp32",
             residual=False),
        # one token through a square projection
        dict(name="gemv_1x4096x4096", op="gemv", tokens=1, n=4096, k=4096, dtype="bf16", layout="mma"),
        # one token through the two stacked MLP input projections of an 8B model
        dict(name="gemv_1x28672x4096", op="gemv", tokens=1, n=28672, k=4096, dtype="bf16", layout="mma_x4"),
        # eight requests decoding together through the MLP output projection
        dict(name="gemv_8x4096x14336", op="gemv", tokens=8, n=4096, k=14336, dtype="bf16", layout="mma"),
        # odd sizes, fp32 activations
        dict(name="gemv_3x1001x2080_f32", op="gemv", tokens=3, n=1001, k=2080, dtype="fp32", layout="plain"),
        # one token through a fused query, key and value projection, one scale domain
        dict(name="gemv_nvfp4_1x6144x4096", op="gemv_nvfp4", tokens=1, n=6144, k=4096, dtype="bf16", layout="mma",
             domain=0),
        # sixteen requests through an MLP projection, a scale domain for each 128 weight rows
        dict(name="gemv_nvfp4_16x14336x4096", op="gemv_nvfp4", tokens=16, n=14336, k=4096, dtype="bf16",
             layout="mma_x4", domain=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_cast", "norm_cast", "norm_backward", "gemv", "gemv", "gemv_nvfp4"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("norm"):
        cols = 32 * _log_int(rng, 4, 512)
        rows = _log_int(rng, 1, max(1, min(16384, 8192 * 4096 // cols)))
        case = dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7)
        if op == "norm_cast":
            case |= dict(fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), layout=rng.choice(["mma", "mma_x4", "plain"]),
                         train=rng.random() < 0.5)
        return case
    k = (32 if op == "gemv" else 16) * _log_int(rng, 8, 512)
    n = _log_int(rng, 33, min(28672, 28672 * 4096 // k))
    case = dict(op=op, tokens=rng.randint(1, 16), n=n, k=k, dtype=dtype,
                layout=rng.choice(["mma", "mma_x4", "plain"]))
    if op == "gemv_nvfp4":
        case["domain"] = rng.choice([0, 32, 128])
    return case


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"].startswith("gemv"):
        m, n, k = case["tokens"], case["n"], case["k"]
        group = 32 if case["op"] == "gemv" else 16
        return {"bytes": n * k // 2 + n * k // group + (m * k + m * n) * e, "flops": 2 * m * n * k}
    r, c, res = case["rows"], case["cols"], case["residual"]
    n = r * c
    if case["op"] == "norm_backward":          # reads dy, h, dres, 1/rms; writes dx; weight and its gradient
        return {"bytes": n * e * (4 if res else 3) + 4 * r + (e + 4) * c, "flops": 9 * n}
    b = n * e * (3 if res else 1) + e * c       # x, and with a residual r and h
    if case["op"] == "norm":
        return {"bytes": b + n * e, "flops": 5 * n}
    b += n + n // 32
    if case["train"]:
        b += n * e + 4 * r
    return {"bytes": b, "flops": 8 * n}


# --- scale layouts: an (outer, blocks) table of bytes as the buffer holds it

def _padded(outer, blocks):
    return (outer + 127) // 128 * 128, (blocks + 3) // 4 * 4


def _scales_size(outer, blocks, layout):
    if layout == "plain":
        return outer * blocks
    ro, kb = _padded(outer, blocks)
    return ro * kb * (4 if layout == "mma_x4" else 1)


def _lay_out(table, layout):
    if layout == "plain":
        return table.reshape(-1)
    outer, blocks = table.shape
    ro, kb = _padded(outer, blocks)
    full = torch.zeros((ro, kb), dtype=table.dtype, device=table.device)
    full[:outer, :blocks] = table
    atoms = full.view(ro // 128, 4, 32, kb // 4, 4).permute(0, 3, 2, 1, 4)
    if layout == "mma_x4":
        atoms = atoms.unsqueeze(2).expand(-1, -1, 4, -1, -1, -1)
    return atoms.reshape(-1)


def _table(buf, outer, blocks, layout):
    if layout == "plain":
        return buf[:outer * blocks].view(outer, blocks)
    ro, kb = _padded(outer, blocks)
    if layout == "mma_x4":
        buf = buf.view(ro * kb // 512, 4, 512)[:, 0]
    atoms = buf.reshape(ro // 128, kb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return atoms.reshape(ro, kb)[:outer, :blocks]


# --- the casts, in elementary operations

def _block_scales(v, fmt):
    """E8M0 scale bytes of (outer, blocks, 32) fp32 values, and the values over their scale."""
    v = torch.where(v.abs() < 2.0 ** -126, torch.zeros_like(v), v)
    amax = v.abs().amax(-1)
    _, ex = torch.frexp(amax)                                   # amax = f 2^ex, f in [1/2, 1)
    e = (ex - 1 - EMAX[fmt]).clamp(-127, 127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    down = ((127 - e).to(torch.int32) << 23).view(torch.float32)  # 2^-e
    return (e + 127).to(torch.uint8), v * down.unsqueeze(-1)


def _e2m1(u):
    """E2M1 code (0..15) nearest to each value, ties to the even code."""
    a = u.abs()
    c = torch.zeros_like(a, dtype=torch.uint8)
    c = c + (a > 0.25) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return c.to(torch.uint8) + 8 * (u < 0).to(torch.uint8)


def _e2m1_value(code):
    m = (code & 7).to(torch.int16)
    q = torch.where(m < 2, 2 * m, (2 + (m & 1)) << (m >> 1))     # four times the magnitude
    return torch.where(code >= 8, -q, q).to(torch.float32) * 0.25


def _pack4(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def _unpack4(packed):
    return torch.stack((packed & 15, packed >> 4), -1).flatten(1)


def _mxfp4_weights(w, layout):
    n, k = w.shape
    s, u = _block_scales(w.view(n, k // 32, 32), "e2m1")
    return _pack4(_e2m1(u).view(n, k)), _lay_out(s, layout).contiguous()


def _nvfp4_weights(w, layout, domain):
    n, k = w.shape
    lines = domain or n
    doms = (n + lines - 1) // lines
    top = torch.zeros((doms * lines,), device=w.device)
    top[:n] = w.abs().amax(1)
    top = top.view(doms, lines).amax(1)
    enc = torch.where(top > 0, 2688.0 / top, torch.ones_like(top))
    e = enc.repeat_interleave(lines)[:n].unsqueeze(1)
    b = w.view(n, k // 16, 16)
    s = ((b.abs().amax(-1) / 6.0) * e).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.to(torch.float32)
    r = torch.where(d > 0, e / d, torch.zeros_like(d))
    codes = _e2m1((b * r.unsqueeze(-1)).clamp(-6.0, 6.0)).view(n, k)
    return _pack4(codes), _lay_out(s.view(torch.uint8), layout).contiguous(), enc.contiguous()


# --- what a program has in hand

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    dt = DTYPE[case["dtype"]]
    s = dict(case)
    if case["op"].startswith("gemv"):
        m, n, k = case["tokens"], case["n"], case["k"]
        s["x"] = normal(m, k).to(dt)
        w = normal(n, k) * 0.02 * torch.exp(0.3 * normal(n, 1))
        if case["op"] == "gemv":
            s["w"] = _mxfp4_weights(w, case["layout"])
        else:
            s["w"] = _nvfp4_weights(w, case["layout"], case["domain"])
        s["y"] = torch.empty((m, n), dtype=dt, device="cuda")
        return s
    r, c = case["rows"], case["cols"]
    loud = torch.where(torch.rand((c,), generator=g, device="cuda") < 0.01, 20.0, 1.0)   # a few loud channels
    stream = normal(r, c) * loud * torch.exp(0.5 * normal(r, 1))
    s["weight"] = (1.0 + 0.1 * normal(c)).to(dt)
    if case["op"] == "norm_backward":
        s["h"] = stream.to(dt)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dy"] = normal(r, c).to(dt)
        s["dres"] = normal(r, c).to(dt) if case["residual"] else None
        s["out"] = (torch.empty_like(s["dy"]), torch.empty((c,), device="cuda"))
        return s
    s["residual"] = stream.to(dt) if case["residual"] else None
    s["x"] = normal(r, c).to(dt) if case["residual"] else stream.to(dt)
    h = torch.empty_like(s["x"]) if case["residual"] else None
    if case["op"] == "norm":
        s["out"] = (torch.empty_like(s["x"]), h, None)
        return s
    codes = torch.empty((r, c), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(_scales_size(r, c // 32, case["layout"]), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(s["x"]) if case["train"] else None
    rstd = torch.empty((r,), device="cuda") if case["train"] else None
    s["out"] = (codes, scales, h, y, rstd)
    return s


# --- one pass

def run(s):
    if own:
        return _call(s)
    return {"norm": _norm, "norm_cast": _norm_cast, "norm_backward": _norm_backward, "gemv": _gemv,
            "gemv_nvfp4": _gemv_nvfp4}[s["op"]](s)


def _call(s):
    from microscaling_block_scaled_mx_b200 import mx
    op = s["op"]
    if op == "gemv":
        return {"y": mx.gemv(*s["w"], s["x"], s["n"], s["k"], out=s["y"], scale_layout=s["layout"])}
    if op == "gemv_nvfp4":
        return {"y": mx.gemv_nvfp4(s["w"], s["x"], s["n"], s["k"], domain_rows=s["domain"], out=s["y"],
                                   scale_layout=s["layout"])}
    if op == "norm_backward":
        dx, dweight = mx.rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dres=s["dres"], out=s["out"])
        return {"dx": dx, "dweight": dweight}
    if op == "norm":
        y, h, _ = mx.rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], out=s["out"])
        return _named(y=y, h=h)
    codes, scales, h, y, rstd = mx.rmsnorm_quantize(
        s["x"], s["weight"], EPS, residual=s["residual"], fmt=s["fmt"], scale_layout=s["layout"],
        with_y=s["train"], with_rstd=s["train"], out=s["out"])
    return _named(codes=codes.view(FLOAT8[s["fmt"]]), scales=scales.view(torch.float8_e8m0fnu), h=h, y=y, rstd=rstd)


def _named(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _norm32(s):
    x, r = s["x"], s["residual"]
    h = None if r is None else (x.float() + r.float()).to(x.dtype)     # kept in x's type, and read back from it
    v = (x if h is None else h).float()
    rstd = 1.0 / torch.sqrt(v.square().mean(1) + EPS)
    return h, v * rstd.unsqueeze(1) * s["weight"].float(), rstd


def _norm(s):
    h, y, _ = _norm32(s)
    return _named(y=y.to(s["x"].dtype), h=h)


def _norm_cast(s):
    h, y, rstd = _norm32(s)
    rows, cols = y.shape
    scales, u = _block_scales(y.view(rows, cols // 32, 32), s["fmt"])
    top = MAXV[s["fmt"]]
    codes = u.clamp(-top, top).view(rows, cols).to(FLOAT8[s["fmt"]])
    keep = s["train"]
    return _named(codes=codes, scales=_lay_out(scales, s["layout"]).view(torch.float8_e8m0fnu), h=h,
                  y=y.to(s["x"].dtype) if keep else None, rstd=rstd if keep else None)


def _norm_backward(s):
    dy, w, rstd = s["dy"].float(), s["weight"].float(), s["rstd"].unsqueeze(1)
    n = s["h"].float() * rstd
    a = dy * w
    dx = rstd * (a - n * (a * n).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * n).sum(0)}


def _gemv(s):
    n, k = s["n"], s["k"]
    packed, buf = s["w"]
    scale = _table(buf, n, k // 32, s["layout"]).contiguous().view(torch.float8_e8m0fnu).to(torch.float32)
    w = (_e2m1_value(_unpack4(packed)).view(n, k // 32, 32) * scale.unsqueeze(-1)).view(n, k)
    return {"y": torch.matmul(s["x"].float(), w.t()).to(s["x"].dtype)}


def _gemv_nvfp4(s):
    n, k = s["n"], s["k"]
    packed, buf, enc = s["w"]
    scale = _table(buf, n, k // 16, s["layout"]).contiguous().view(torch.float8_e4m3fn).to(torch.float32)
    w = (_e2m1_value(_unpack4(packed)).view(n, k // 16, 16) * scale.unsqueeze(-1)).view(n, k)
    e = enc.repeat_interleave(s["domain"] or n)[:n]
    return {"y": (torch.matmul(s["x"].float(), w.t()) / e).to(s["x"].dtype)}


# --- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("gemv"):
        n, k = case["n"], case["k"]
        group = 32 if case["op"] == "gemv" else 16
        values = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                              device="cuda")
        w = torch.empty((n, k), dtype=torch.float64, device="cuda")
        w[:, 0::2] = values[(s["w"][0] & 15).long()]
        w[:, 1::2] = values[(s["w"][0] >> 4).long()]
        b = _table(s["w"][1], n, k // group, case["layout"]).long()
        if case["op"] == "gemv":
            f = torch.pow(torch.full_like(b, 2.0, dtype=torch.float64), b - 127)
        else:
            exp, man = b >> 3, (b & 7).double()
            f = torch.where(exp == 0, man / 512, (1 + man / 8) * torch.pow(2.0, (exp - 7).double()))
            at = torch.arange(n, device="cuda") // (case["domain"] or n)
            f = f / s["w"][2].double()[at].unsqueeze(1)
        w = (w.view(n, k // group, group) * f.unsqueeze(-1)).view(n, k)
        return {"y": s["x"].double() @ w.t()}
    weight = s["weight"].double()
    if case["op"] == "norm_backward":
        h, dy = s["h"].double(), s["dy"].double()
        rstd = s["rstd"].double().unsqueeze(1)
        g = dy * weight
        inner = (g * h).sum(1, keepdim=True) / case["cols"]
        dx = g * rstd - h * inner * rstd ** 3
        if case["residual"]:
            dx = dx + s["dres"].double()
        return {"dx": dx, "dweight": (dy * h * rstd).sum(0)}
    h = s["x"].double()
    if case["residual"]:
        h = (h + s["residual"].double()).to(DTYPE[case["dtype"]]).double()
    rstd = (h.pow(2).sum(1) / case["cols"] + EPS).pow(-0.5)
    y = h * rstd.unsqueeze(1) * weight
    kept = h if case["residual"] else None
    if case["op"] == "norm":
        return _named(y=y, h=kept)
    fmt = case["fmt"]
    blocks = y.view(case["rows"], case["cols"] // 32, 32)
    e = torch.floor(torch.log2(blocks.abs().amax(-1).clamp(min=2.0 ** -200))) - EMAX[fmt]
    e = e.clamp(-127, 127)
    u = blocks / torch.pow(2.0, e).unsqueeze(-1)
    step = torch.pow(2.0, torch.floor(torch.log2(u.abs().clamp(min=2.0 ** EMIN[fmt]))) - MANT[fmt])
    codes = (torch.round(u / step) * step).clamp(-MAXV[fmt], MAXV[fmt]).view_as(y)
    scales = torch.pow(2.0, _lay_out(e + 127, case["layout"]) - 127)
    keep = case["train"]
    return _named(codes=codes, scales=scales, h=kept, y=y if keep else None, rstd=rstd if keep else None)
