"""The product's GELU at every bf16 and between them, in both types of result: within its bound, and bf16 the rounding of
binary32."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 40, 3000])
@pytest.mark.parametrize("cut", [0, 1])
def test_every_bf16(m, cut):
    """Given by the bias of a product with an empty k; cut: a width that holds no vectors."""
    dev = torch.device("cuda:0")
    every = torch.arange(65536, dtype=torch.int32, device=dev).to(torch.int16).view(torch.bfloat16).float()
    z = torch.cat((torch.linspace(-12, 12, 4096, device=dev)[cut:], every))
    n = z.numel()
    a, b = torch.empty((m, 0), dtype=torch.uint8, device=dev), torch.empty((n, 0), dtype=torch.uint8, device=dev)
    d, y = torch.empty((m, n), device=dev), torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    fp8q.fp8q_matmul(a, b, d, bias=z, act=1)
    fp8q.fp8q_matmul(a, b, y, bias=z, act=1)
    nan = z.isnan() | (z == -float("inf"))
    assert torch.equal(d.isnan(), nan.expand(m, n)) and torch.equal(y.isnan(), nan.expand(m, n))
    d, y, x = d[:, ~nan], y[:, ~nan], z[~nan].double()
    assert torch.equal(y, d.to(torch.bfloat16)), "bf16 is not the rounding of the float32 result"
    assert (d == d[:1]).all()
    u = -2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)
    want = torch.where(x < -30, torch.zeros_like(x), torch.where(x > 30, x, x / (1 + torch.exp(u))))
    near = x.abs() < 5  # where 1 + tanh keeps its digits: the tests' other form of the definition
    assert ((R.gelu(x) - want).abs() <= 2.0 ** -30 * want.abs())[near].all()
    rel = torch.where(x >= -5, 2.0 ** -18, 2.0 ** -16)
    bound = torch.where(x >= -10, rel * want.abs() + 2.0 ** -130, torch.full_like(x, 2.0 ** -100))
    fine = x.isfinite()
    assert ((d[0].double() - want).abs() <= bound)[fine].all()
    assert (d[0][~fine] == float("inf")).all()
