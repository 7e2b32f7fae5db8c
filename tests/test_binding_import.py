"""The binding on a torch that lacks the CUDA build's private helpers: it
imports, and its checks and size functions work, as where they exist."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_HELPERS = """
import sys
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
sys.path.insert(0, {root!r})
from microscaling_block_scaled_mx_b200 import mx
assert mx.codes_row_bytes("e2m1", 64) == 32
x, w = torch.zeros(4, 64), torch.zeros(64)
for call in (lambda: mx.rmsnorm(x, w), lambda: mx.gemv(x, x, x, 16, 64)):
    try:
        call()
    except ValueError as e:
        assert "CUDA device" in str(e)
    else:
        raise AssertionError("a CPU tensor was taken")
# the public functions stand in for the helpers
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device: type("Stream", (), dict(cuda_stream=100 + device))
assert mx._current_device() == 3 and mx._handle(None, 5) == 105
"""


def test_binding_without_private_helpers():
    r = subprocess.run([sys.executable, "-c", WITHOUT_HELPERS.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
