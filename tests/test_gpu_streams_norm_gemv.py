"""GPU tests of the norm and the 4-bit products on several streams that wait for
one another, eager and captured: a call starts while its stream's last kernel
drains, and must still see what every stream that it waits for has written.
The same calls one at a time, with the device waited for, give the bits."""
import pytest
import torch

from gpu_helpers import dev
from microscaling_block_scaled_mx_b200 import mx
from test_gpu_gemv import activations, mx_weights, nv_weights

pytestmark = pytest.mark.gpu

K = 2048


@pytest.fixture(scope="module")
def state():
    codes, scales, _ = mx_weights(K, K, "mma", 1, 114, 120)
    ws, _ = nv_weights(K, K, "mma_x4", 0, 2)
    w = torch.ones(K, device=dev()).bfloat16()
    return dict(codes=codes, scales=scales, ws=ws, w=w, x=activations(3, K, torch.bfloat16, 3),
                big=activations(400, K, torch.bfloat16, 4), ws_back=mx.rmsnorm_backward_workspace(400, K))


def forked(s, side, wait):
    """Both streams read what the other wrote, five times over; `wait` ends each step."""
    main = torch.cuda.current_stream()
    y, h, _ = mx.rmsnorm(s["x"], s["w"], residual=s["x"])
    out = []
    for _ in range(5):
        wait()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a = mx.gemv(s["codes"], s["scales"], y, K, K)           # behind main's norm
            wait()
            q, qs, qh, _, rstd = mx.rmsnorm_quantize(s["big"], s["w"], residual=s["big"], with_rstd=True, scale_layout="plain")
            wait()
            dx, dw = mx.rmsnorm_backward(s["big"], qh, s["w"], rstd, dres=qh, workspace=s["ws_back"])
        b = mx.gemv_nvfp4(s["ws"], y, K, K, scale_layout="mma_x4")
        wait()
        main.wait_stream(side)
        y, h, _ = mx.rmsnorm(a, s["w"], residual=b)                  # behind both
        wait()
        z = mx.gemv(s["codes"], s["scales"], (dx[:3] + y).contiguous(), K, K)
        out += [a, b, y, h, q, qs, rstd, dx, dw, z]
    return out


def test_eager(state):
    side = torch.cuda.Stream()
    want = [t.clone() for t in forked(state, side, torch.cuda.synchronize)]
    torch.cuda.synchronize()
    keep = []                                   # no memory goes from one stream to the other meanwhile
    for _ in range(10):
        got = forked(state, side, lambda: None)
        keep.append(got)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured(state):
    side = torch.cuda.Stream()
    want = [t.clone() for t in forked(state, side, torch.cuda.synchronize)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = forked(state, side, lambda: None)
    for _ in range(10):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_of_the_same_calls(state):
    """Each with a workspace of its own, replayed on two streams at once."""
    h, rstd = state["big"], mx.rmsnorm(state["big"], state["w"], with_rstd=True)[2]
    want = mx.rmsnorm_backward(h, h, state["w"], rstd, dres=h)
    y_want = mx.gemv(state["codes"], state["scales"], state["x"], K, K)
    graphs, outs = [], []
    for _ in range(2):
        ws = mx.rmsnorm_backward_workspace(400, K)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                dx, dw = mx.rmsnorm_backward(h, h, state["w"], rstd, dres=h, workspace=ws)
                y = mx.gemv(state["codes"], state["scales"], state["x"], K, K)
        graphs.append(g)
        outs.append((dx, dw, y, ws))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for dx, dw, y, _ in outs:
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and torch.equal(y, y_want)
