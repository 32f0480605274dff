"""Tensors of a float8 type whose format is not the one that a call names are refused, and read right where it is."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_matmul import check, gen

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def refused(f, what):
    with pytest.raises(ValueError, match=what):
        f()


def test_products(dev):
    g = gen(dev, 1)
    a, b, w = R.random_codes((40, 64), 1, g).view(E5), R.random_codes((32, 64), 0, g).view(E4), R.random_codes((2, 32, 64), 0, g).view(E4)
    d, q, one = torch.empty((40, 32), device=dev), torch.zeros((40, 32), dtype=torch.uint8, device=dev), torch.ones(1, device=dev)
    at = torch.tensor([0, 10, 40], dtype=torch.int32, device=dev)
    refused(lambda: fp8q.fp8q_matmul(a, b, d), "a has dtype")  # e5m2 codes under the default e4m3
    refused(lambda: fp8q.fp8q_matmul(a, b, d, 1, 1), "b has dtype")
    refused(lambda: fp8q.fp8q_grouped_matmul(a, w, at, d), "a has dtype")
    refused(lambda: fp8q.fp8q_grouped_matmul(a, w, at, d, 1, 1), "b has dtype")
    for fmt, t in ((0, E5), (1, E4)):
        refused(lambda: fp8q.fp8q_matmul(a, b, None, 1, 0, q=q.view(t), q_fmt=fmt, q_scale=one), "q has dtype")
    h, sf = fp8q.checkpoint_empty(40, 32)
    refused(lambda: fp8q.fp8q_matmul(a, b, None, 1, 0, h=h.view(E5), h_sf=sf), "h has dtype")
    dw, back = torch.empty((2, 64, 32), device=dev), R.random_codes((40, 32), 0, g).view(E4)
    refused(lambda: fp8q.fp8q_grouped_weight_gradient(a, back.view(torch.uint8).view(E5), at, dw), "b has dtype")
    refused(lambda: fp8q.fp8q_grouped_weight_gradient(a, back, at, dw, 0, 0), "a has dtype")
    assert not q.any()
    # the right ones, and bytes under any format
    va, vb = a.float().double(), b.float().double()
    for x, y in ((a, b), (a.view(torch.uint8), b.view(torch.uint8)), (a.view(torch.uint8), b)):
        fp8q.fp8q_matmul(x, y, d, 1, 0, q=None)
        check(d, va @ vb.t(), R.sum_bound(va, vb))
    fp8q.fp8q_matmul(a, b, None, 1, 0, q=q.view(E5), q_fmt=1, q_scale=one, h=h.view(E4), h_sf=sf)
    fp8q.fp8q_grouped_weight_gradient(a, back, at, dw)
    v = back.float().double()
    check(dw[1], va[10:].t() @ v[10:], R.sum_bound(va[10:].t(), v[10:].t()))


def test_checkpoints(dev):
    x, y = torch.randn((8, 64), device=dev).bfloat16(), torch.empty((8, 64), dtype=torch.bfloat16, device=dev)
    h, sf = fp8q.checkpoint_empty(8, 64)
    one, q = torch.ones(1, device=dev), torch.empty((8, 64), dtype=torch.uint8, device=dev)
    refused(lambda: fp8q.fp8q_checkpoint_quantize(x, h.view(E5), sf), "q has dtype")
    fp8q.fp8q_checkpoint_quantize(x, h.view(E4), sf)
    refused(lambda: fp8q.fp8q_checkpoint_dequantize(h.view(E5), sf, y), "q has dtype")
    fp8q.fp8q_checkpoint_dequantize(h.view(E4), sf, y)
    back = lambda h, q, fmt: fp8q.fp8q_gelu_backward_quantize_amax(x, h, sf, q, fmt, one)  # noqa: E731
    refused(lambda: back(h.view(E5), q, 1), "h has dtype")
    refused(lambda: back(h, q.view(E4), 1), "q has dtype")
    refused(lambda: back(h, q.view(E5), 0), "q has dtype")
    back(h.view(E4), q.view(E5), 1)
    back(h.view(E4), q.view(E4), 0)
