"""Waits of the FP8 products that run out, without any fault: the library built once more with its test hooks, in which one
wait, of one role at one step, reports failure in a single lane of its warp although what it waits for has come.  The call
has to end, with NaN or the right value in every element, and the device has to be as usable as before."""
import ctypes

import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_matmul import gen

pytestmark = pytest.mark.gpu

COPY_EMPTY, SUM_FULL, SUM_DRAINED, MASK_FULL, OUT_DONE = range(1, 6)


@pytest.fixture
def hooked(hooks_lib):
    hooks_lib.fp8q_matmul.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    hooks_lib.fp8q_grouped_weight_gradient.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    hooks_lib.fp8q_test_set_product_give_up.argtypes = [ctypes.c_int] * 3
    hooks_lib.fp8q_test_set_product_give_up.restype = None
    yield hooks_lib
    hooks_lib.fp8q_test_set_product_give_up(0, 0, -1)


def check(hooked, f, want, got, role, at, cta):
    """f(lib) runs the call into got."""
    hooked.fp8q_test_set_product_give_up(role, at, cta)
    assert f(hooked) == 0
    torch.cuda.synchronize()  # the call ends: nothing waits forever
    lost = torch.isnan(got)
    assert torch.equal(got[~lost], want[~lost]), "an element that is neither right nor NaN"
    hooked.fp8q_test_set_product_give_up(0, 0, -1)
    got.zero_()
    assert f(hooked) == 0
    torch.cuda.synchronize()
    assert torch.equal(got, want), "the same kernel behind one that gave up"
    return lost


def product(m, n, k, dtype, ta=0):
    dev = torch.device("cuda:0")
    g = gen(dev, 1)
    a, b = R.random_codes((k, m) if ta else (m, k), 0, g), R.random_codes((n, k), 0, g)
    want = torch.empty((m, n), dtype=dtype, device=dev)
    fp8q.fp8q_matmul(a, b, want, a_trans=ta)
    got = torch.zeros_like(want)
    p = fp8q.Product(m=m, n=n, k=k, a=a.data_ptr(), b=b.data_ptr(), lda=a.shape[1], ldb=k, a_trans=ta, d=got.data_ptr(), out=int(dtype == torch.float32))
    keep = (a, b)
    return lambda lib: (keep, lib.fp8q_matmul(ctypes.byref(p), torch.cuda.current_stream().cuda_stream))[1], want, got


@pytest.mark.parametrize("role,at", [(COPY_EMPTY, 0), (COPY_EMPTY, 1), (SUM_FULL, 0), (SUM_FULL, 1), (OUT_DONE, 0)])
@pytest.mark.parametrize("m,n,k,ta", [(1, 640, 8192, 0), (40, 256, 8192, 0), (65, 200, 1040, 0), (304, 520, 1280, 1)])
def test_single_ctas(hooked, m, n, k, ta, role, at):
    f, want, got = product(m, n, k, torch.bfloat16, ta)
    assert check(hooked, f, want, got, role, at, -1).all()
    f, want, got = product(m, n, k, torch.float32, ta)
    lost = check(hooked, f, want, got, role, at, 1)
    assert lost.any() and int(lost.sum()) <= 128 * 128


@pytest.mark.parametrize("role,at", [(COPY_EMPTY, 0), (COPY_EMPTY, 7), (SUM_FULL, 0), (SUM_FULL, 1), (SUM_FULL, 6), (SUM_FULL, 9), (SUM_DRAINED, 2),
                                     (OUT_DONE, 0), (OUT_DONE, 1), (OUT_DONE, 2)])
@pytest.mark.parametrize("m,n", [(4400, 2304), (4300, 2751)])
def test_pairs(hooked, m, n, role, at):
    """Pairs of CTAs, the first of which take three tiles of 256 x 256, 5 steps each."""
    for dtype, cta in ((torch.bfloat16, -1), (torch.float32, 0), (torch.bfloat16, 1)):
        if cta == 1 and role in (SUM_FULL, SUM_DRAINED):
            continue  # the first CTA of a pair issues for both
        f, want, got = product(m, n, 560, dtype)
        lost = check(hooked, f, want, got, role, at, cta)
        assert lost.any() and (cta < 0 or int(lost.sum()) <= 3 * 256 * 256)


@pytest.mark.parametrize("role,at", [(COPY_EMPTY, 0), (COPY_EMPTY, 2), (MASK_FULL, 0), (MASK_FULL, 2), (SUM_FULL, 1), (OUT_DONE, 0)])
def test_weight_gradients(hooked, role, at):
    dev = torch.device("cuda:0")
    g = gen(dev, 2)
    a, b = R.random_codes((700, 528), 0, g), R.random_codes((700, 304), 0, g)
    off = torch.tensor([0, 300, 300, 333, 700], dtype=torch.int32, device=dev)
    want = torch.empty((4, 528, 304), device=dev)
    fp8q.fp8q_grouped_weight_gradient(a, b, off, want, 0, 0)
    got = torch.zeros_like(want)
    p = fp8q.Product(m=528, n=304, k=700, a=a.data_ptr(), b=b.data_ptr(), lda=528, ldb=304, a_trans=1, b_trans=1, d=got.data_ptr(), out=1)
    f = lambda lib: lib.fp8q_grouped_weight_gradient(ctypes.byref(p), off.data_ptr(), 4, torch.cuda.current_stream().cuda_stream)  # noqa: E731
    for cta in (-1, 0):
        assert check(hooked, f, want, got, role, at, cta).any()
