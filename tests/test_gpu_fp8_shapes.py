"""Outputs and epilogue inputs of the right number of elements in rows of another length are refused: they would be filled in
the wrong order.  Leading dimensions may be split or flattened."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_matmul import gen, stored

pytestmark = pytest.mark.gpu
M, N, K = 24, 64, 32


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def bf(*s):
    return torch.full(s, 5.0, dtype=torch.bfloat16, device="cuda")


def u8(*s):
    return torch.full(s, 9, dtype=torch.uint8, device="cuda")


def f32(*s):
    return torch.full(s, 3.0, device="cuda")


@pytest.mark.parametrize("grouped", [False, True])
def test_products(dev, grouped):
    g = gen(dev, 1)
    a, w = R.random_codes((M, K), 0, g), R.random_codes((2, N, K), 0, g)
    at, one = torch.tensor([0, 10, M], dtype=torch.int32, device=dev), f32(1)
    call = (lambda **o: fp8q.fp8q_grouped_matmul(a, w, at, q_scale=one, **o)) if grouped else (lambda **o: fp8q.fp8q_matmul(a, w[0], q_scale=one, **o))
    good = dict(d=bf(M, N), residual=bf(M, N), q=u8(M, N), h=u8(M, N), h_sf=u8(M, 2), bias=f32(2, N) if grouped else f32(N))
    for name, wrong in (("d", bf(N, M)), ("residual", bf(N, M)), ("q", u8(N, M)), ("h", u8(N, M)), ("h_sf", u8(2, M)), ("h_sf", u8(1, 2 * M)), ("d", bf(2, N // 2, M)),
                        *((("bias", f32(N, 2)),) if grouped else (("bias", f32(N, 1)),))):
        with pytest.raises(ValueError, match=f"{name} must be"):
            call(**{**good, name: wrong})
    assert (good["d"] == 5).all() and (good["q"] == 9).all()
    call(**good)
    split = {k: t.clone().reshape(2, M // 2, -1) if k != "bias" else t for k, t in good.items()}
    flat = {k: t.clone().reshape(-1) for k, t in good.items()}
    call(**split), call(**flat)
    for k in ("d", "q", "h", "h_sf"):
        assert torch.equal(split[k].view_as(good[k]), good[k]) and torch.equal(flat[k].view_as(good[k]), good[k])


def test_weight_gradients(dev):
    g = gen(dev, 2)
    a, b, at = stored(R.random_codes((40, M), 1, g), 0), R.random_codes((40, N), 0, g), torch.tensor([0, 10, 40], dtype=torch.int32, device=dev)
    d = f32(2, M, N)
    for wrong in (f32(2, N, M), f32(M, 2, N), f32(2 * N, M)):
        with pytest.raises(ValueError, match="residual must be"):
            fp8q.fp8q_grouped_weight_gradient(a, b, at, d, residual=wrong)
    assert (d == 3).all()
    flat = torch.empty_like(d)
    fp8q.fp8q_grouped_weight_gradient(a, b, at, flat, residual=f32(2 * M, N))
    fp8q.fp8q_grouped_weight_gradient(a, b, at, d, residual=d)
    assert torch.equal(d, flat)


def test_checkpoints(dev):
    x, q, sf = torch.randn((M, N), device=dev).bfloat16(), u8(M, N), u8(M, 2)
    for wrong in (dict(q=u8(N, M)), dict(sf=u8(2, M))):
        with pytest.raises(ValueError):
            fp8q.fp8q_checkpoint_quantize(**{**dict(x=x, q=q, sf=sf), **wrong})
    fp8q.fp8q_checkpoint_quantize(x, q.view(2, M // 2, N), sf.view(-1))
    with pytest.raises(ValueError):
        fp8q.fp8q_checkpoint_dequantize(q.view(N, M), sf, x)
    good = dict(d_y=x, h=q, h_sf=sf, q=u8(M, N), d_x=bf(M, N), d_bias=f32(N), scale=f32(1), workspace=u8(fp8q.gelu_backward_workspace(M, N) + 16))
    for wrong in (dict(h=q.view(N, M)), dict(h_sf=sf.view(2, M)), dict(q=u8(N, M)), dict(d_x=bf(N, M)), dict(d_bias=f32(N, 1))):
        with pytest.raises(ValueError):
            fp8q.fp8q_gelu_backward_quantize_amax(**{**good, **wrong})
    assert (good["d_x"] == 5).all()
    fp8q.fp8q_gelu_backward_quantize_amax(**good)
    assert not (good["d_x"] == 5).all()
