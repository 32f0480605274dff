"""Sums over so long a k that a tile takes longer than a wait may: the library built once more with its test hooks, whose
waits give up after a tenth of a second.  Codes of 1 and -1, so that every sum is a whole number that binary32 holds."""
import ctypes

import pytest
import torch

from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_matmul import gen

pytestmark = pytest.mark.gpu
M = 16


def signs(shape, dev, seed):
    """Codes of 1 and -1."""
    return torch.empty(shape, dtype=torch.uint8, device=dev).random_(0, 2, generator=gen(dev, seed)).mul_(0x80).add_(0x38)


def sums(a, b, step=1 << 22):
    """[m, n] of a [m, k] and b [n, k], exactly: parts of k whose sums are below 2^24, added in 64 bits."""
    v = lambda t: t.contiguous().view(torch.float8_e4m3fn).float()  # noqa: E731
    return sum((v(a[:, i: i + step]) @ v(b[:, i: i + step]).t()).double() for i in range(0, a.shape[1], step))


def took(f):
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    assert f() == 0
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end)


def test_weight_gradients(hooks_lib):
    dev = torch.device("cuda:0")
    rows = 160_000_000
    f = hooks_lib.fp8q_grouped_weight_gradient
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    a, b = signs((rows, M), dev, 1), signs((rows, M), dev, 2)
    off = torch.tensor([0, 1000, rows], dtype=torch.int32, device=dev)
    d = torch.zeros((2, M, M), device=dev)
    p = fp8q.Product(m=M, n=M, k=rows, a=a.data_ptr(), b=b.data_ptr(), lda=M, ldb=M, a_trans=1, b_trans=1, d=d.data_ptr(), out=1)
    ms = took(lambda: f(ctypes.byref(p), off.data_ptr(), 2, torch.cuda.current_stream().cuda_stream))
    assert ms > 200, "no longer than a wait may take: more rows"
    for i, (lo, hi) in enumerate(((0, 1000), (1000, rows))):
        assert torch.equal(d[i].double(), sums(a[lo:hi].t(), b[lo:hi].t()))


def test_single_ctas(hooks_lib):
    dev = torch.device("cuda:0")
    k = 3 << 29
    f = hooks_lib.fp8q_matmul
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    a = signs((M, k + 16), dev, 3)
    d = torch.zeros((M, M), device=dev)
    p = fp8q.Product(m=M, n=M, k=k, a=a.data_ptr(), b=a.data_ptr() + 16, lda=k + 16, ldb=k + 16, d=d.data_ptr(), out=1)
    ms = took(lambda: f(ctypes.byref(p), torch.cuda.current_stream().cuda_stream))
    assert ms > 150, "no longer than a wait may take: a longer k"
    assert torch.equal(d.double(), sums(a[:, :k], a[:, 16:]))
