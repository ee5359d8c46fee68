"""The bounded waits of the tensor-core kernels' header (csrc/cq_tensor.cuh), in a kernel
of the test's own: one barrier gets no arrival, the wait for it runs out, every
role leaves its loop, and the report is there once."""
import ctypes
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def roles(tmp_path_factory):
    from minimax_scale_search_b200 import build
    out = str(tmp_path_factory.mktemp("waits") / "wait_limit.so")
    subprocess.run([build.nvcc(), "-shared", "-O3", "-std=c++17", *build.ARCH, "-Xcompiler", "-fPIC", "-I",
                    os.path.join(build.PKG, "csrc"), "-o", out, os.path.join(HERE, "wait_limit.cu")], check=True)
    lib = ctypes.CDLL(out)
    lib.run_roles.argtypes = [ctypes.c_uint64, ctypes.c_int, ctypes.c_void_p]
    return lib


def run(lib, lost, most=1_000_000):
    import torch
    left = torch.zeros(3, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert lib.run_roles(most, lost, left.data_ptr()) == 0
    return left.tolist()


def reported(lib):
    gave_up = ctypes.c_int(-1)
    assert lib.reported(ctypes.byref(gave_up)) == 0
    return gave_up.value


def test_a_wait_that_runs_out_is_reported_once(roles):
    assert run(roles, lost=-1) == [4, 4, 4] and reported(roles) == 0
    # role 1 does not let role 2 go in its second round: role 2 gives up there, role 0 a round later, role 1 after that
    assert run(roles, lost=1) == [-3, -3, -2]
    assert reported(roles) == 1
    assert reported(roles) == 0  # told once
    assert run(roles, lost=-1) == [4, 4, 4] and reported(roles) == 0


def test_status_is_fine_after_calls_of_every_kind():
    import torch
    from minimax_scale_search_b200 import cq
    zeros = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    w = cq.w4_weights(cq.GPTQTensors(zeros(64, 264), zeros(4, 33), zeros(4, 264, dtype=torch.float16),
                                     torch.arange(512, dtype=torch.int32, device="cuda") // 128))
    for T in (1, 12, 40, 700):
        x, dz = zeros(T, 512, dtype=torch.bfloat16), zeros(T, 264, dtype=torch.bfloat16)
        cq.w4_linear(x, w)
        cq.w4_linear_backward(dz, x, w)
        assert cq.w4_status() == cq.CQ_OK
