"""The largest values of an 8-bit checkpoint: which finite ones come back infinite, and that all others stay within the
stated bound, from every call that makes a checkpoint."""
import numpy as np
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q

FIRST = 0x7F78  # 248 * 2^120


def patterns():
    """Finite bf16 patterns of the last two binades, both signs."""
    p = np.arange(0x7E80, 0x7F80, dtype=np.uint16)
    return np.concatenate([p, p | 0x8000])


def value(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def within(bits, back):
    """back: what each pattern, a block's largest, comes back as (float64)."""
    infinite = (bits & 0x7FFF) >= FIRST
    x = value(bits)
    assert np.array_equal(np.isinf(back), infinite) and (np.sign(back) == np.sign(x)).all()
    assert (np.abs(back - x) <= np.abs(x) / 16)[~infinite].all()


def test_reference():
    bits = np.zeros((512, 32), np.uint16)
    bits[:, 0] = patterns()
    within(bits[:, 0], R.checkpoint(bits)[2][:, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [1, 16, 31, 32])
def test_calls(cols):
    dev = torch.device("cuda:0")
    bits = patterns()
    x = torch.zeros((512, cols), dtype=torch.bfloat16, device=dev)
    x[:, 0] = torch.from_numpy(bits.view(np.int16)).to(dev).view(torch.bfloat16)
    h, sf = fp8q.checkpoint_empty(512, cols)
    y = torch.empty_like(x)
    fp8q.fp8q_checkpoint_quantize(x, h, sf)
    fp8q.fp8q_checkpoint_dequantize(h, sf, y)
    within(bits, y[:, 0].double().cpu().numpy())
    assert not y[:, 1:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 300])
@pytest.mark.parametrize("n", [16384, 16383])
def test_products(m, n):
    """The same from a product's epilogue, whose bias is the value: every 32nd column a pattern."""
    dev = torch.device("cuda:0")
    bits = patterns()
    bias = torch.zeros(512, 32, device=dev)
    bias[:, 0] = torch.from_numpy(value(bits)).to(dev).float()
    bias = bias.view(-1)[:n].contiguous()
    a, b = torch.empty((m, 0), dtype=torch.uint8, device=dev), torch.empty((n, 0), dtype=torch.uint8, device=dev)
    h, sf = fp8q.checkpoint_empty(m, n)
    y = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    fp8q.fp8q_matmul(a, b, None, bias=bias, h=h, h_sf=sf)
    fp8q.fp8q_checkpoint_dequantize(h, sf, y)
    for row in (0, m - 1):
        within(bits, y[row, ::32].double().cpu().numpy())
