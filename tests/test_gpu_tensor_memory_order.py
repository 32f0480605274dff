"""The 4-bit product beside kernels that take tensor memory themselves, in one stream, starts and ends overlapping.

A kernel that holds tensor memory while it waits for the kernel ahead can keep that one from the tensor memory it needs
to end.  The product takes its own behind its wait, and lets the next kernel start only then, so neither neighbour can
be kept waiting, whatever order it takes its own in."""
import ctypes
import os
import subprocess

import pytest
import torch

import fp4_reference as R
from conftest import ROOT
from quantize_amax_scaling_gb300 import build, fp8q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def neighbour(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("neighbours") / "libneighbours.so")
    subprocess.run([build.nvcc_path(), *build.ARCH, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-o", so,
                    os.path.join(ROOT, "tests", "csrc", "tensor_memory_neighbours.cu")], check=True)
    f = ctypes.CDLL(so).launch_neighbour
    f.argtypes, f.restype = [ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int
    return f


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (24, 6000, 4096), (300, 520, 320), (2560, 2304, 1100)])
def test_between_neighbours(neighbour, m, n, k, fmt):
    dev = torch.device("cuda:0")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device=dev)
    g.manual_seed(k)
    ops = []
    for r in (m, n):
        q, s = fp8q.fp4_empty(r, k, fmt)
        ops += [q.random_(0, 256, generator=g), s.fill_(127 if fmt == R.MXFP4 else 0x38)]
    want = torch.empty((m, n), device=dev)
    fp8q.fp8q_fp4_matmul(*ops, want, k, fmt)
    got = [torch.zeros_like(want) for _ in range(3)]
    count = torch.zeros(1, dtype=torch.int64, device=dev)
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    for d in got:
        assert neighbour(0, sms, count.data_ptr(), side.cuda_stream) == 0
        fp8q.fp8q_fp4_matmul(*ops, d, k, fmt, stream=side)
        assert neighbour(1, sms, count.data_ptr(), side.cuda_stream) == 0
        fp8q.fp8q_fp4_matmul(*ops, d, k, fmt, stream=side)
    side.synchronize()
    assert int(count) == 6 * sms
    for d in got:
        assert torch.equal(d, want)
