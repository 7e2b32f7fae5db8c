"""How mx_gemv cuts its work, on the CPU: its launcher linked with a fake CUDA
runtime.  The parts of K follow from how many clusters the device holds, and
decide a token's bits, so a query that fails is an error, and the answer is one
for all calls, whichever comes first."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from microscaling_block_scaled_mx_b200 import build as B
    B.build()
    tmp = tmp_path_factory.mktemp("gemv_launch")
    obj = os.path.join(B.PKG, "_build", "mx_gemv.o")
    src = os.path.join(B.CSRC, "mx_gemv.cu")
    if not os.path.exists(obj) or os.path.getmtime(obj) < os.path.getmtime(src):
        obj = str(tmp / "mx_gemv.o")
        subprocess.run([B.nvcc(), *B.NVCC_FLAGS, "-I", B.INCLUDE, "-I", B.CSRC, "-c", src, "-o", obj], check=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc()))), "include")
    exe = str(tmp / "gemv_launch")
    # -no-pie: a kernel has the same address in every run
    subprocess.run(["g++", "-std=c++17", "-O1", "-no-pie", "-I", B.INCLUDE, "-I", B.CSRC, "-I", cuda,
                    os.path.join(HERE, "gemv_launch.cpp"), obj, "-o", exe], check=True)

    def call(*calls):
        r = subprocess.run([exe, *(",".join(map(str, c)) for c in calls)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        *lines, who = r.stdout.split("\n")[:-1]
        return [tuple(line.split()) for line in lines], int(who)
    return call


OK, FAIL = 0, 1
SIZES = [(1, 256, 16384), (3, 777, 5120), (8, 4096, 14336), (16, 300, 8192), (16, 14336, 4096)]
UNASKED = [(1, 4096, 4096), (1, 33, 96), (3, 70000, 1024)]           # bf16: no cluster comes into question


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("f32,nv", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_a_failed_query_is_an_error(run, m, n, k, f32, nv):
    """Nothing is launched, and the next call is as if the failed one had not been."""
    call = (m, n, k, f32, nv)
    (first,), asked = run((*call, OK))
    assert first[0] == "0" and first[1] == "1"
    assert asked != 0                                   # these sizes depend on the answer
    (failed, again), _ = run((*call, FAIL), (*call, OK))
    assert failed[0] != "0" and failed[1] == "0"
    assert again == first


def test_one_answer_whichever_call_comes_first(run):
    """The kernel that is asked is the same one, and every call is launched as it
    is when it comes first."""
    calls = [(m, n, k, f32, nv, OK) for m, n, k in SIZES + UNASKED for f32 in (0, 1) for nv in (0, 1)]
    alone = [run(c) for c in calls]
    together, who = run(*calls)
    backwards, who_back = run(*calls[::-1])
    assert together == [lines[0] for lines, _ in alone] == backwards[::-1]
    assert {who, who_back, *(w for _, w in alone)} <= {who, 0} and who > 0
