"""Tensor scales of the 16-block format where its arithmetic changes: the quotients are exact products with a
reciprocal for scales from 2^-50 to 2^50 and divisions elsewhere, and the largest elements are divided in either
case.  Every bf16, in each of the kernels that quantize: rows on 32-byte boundaries, both directions at once, and rows
that start anywhere; and the norms that quantize their output."""
import numpy as np
import pytest
import torch

import fp4_reference as R
import oracle
from gpu_helpers import assert_codes_equal, bf16_bits_of
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp4 import check_packed, from_bits, guarded_pair

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def f32(v):
    return float(np.float32(v))


def step(v, to):
    return float(np.nextafter(np.float32(v), np.float32(to)))


LO, HI = 2.0 ** -50, 2.0 ** 50
EDGES = [LO, step(LO, 0), step(LO, 1), HI, step(HI, np.inf), step(HI, 0)]
AWKWARD = [f32(s * e) for e in (2.0 ** -49, 2.0 ** -30, 1.0, 2.0 ** 30, 2.0 ** 49)
           for s in (1.9999999, 1.0000001, 4 / 3, 1.0 / 2688 * 2048, 1.4142135)]
OTHER = [2.0 ** -64, 2.0 ** 62, 1e-38, 1e-44, 3e37, 1e38, 0.0, -1.0, float("inf"), float("nan")]


def every_bf16(rows, cols, seed):
    """All bf16 but NaN, neighbours (which share a block) in one half of the rows and in any order in the other."""
    b = np.arange(65536, dtype=np.uint16)
    b = b[(b & 0x7FFF) <= 0x7F80]
    x = np.resize(b, (rows // 2, cols))
    y = np.resize(np.random.RandomState(seed).permutation(b), (rows - rows // 2, cols))
    return np.concatenate([x, y])


@pytest.mark.parametrize("cols", [512, 519])  # rows on 32-byte boundaries, and anywhere
@pytest.mark.parametrize("scale", EDGES + AWKWARD + OTHER)
def test_every_bf16(dev, scale, cols):
    bits = every_bf16(260, cols, 1)
    x = from_bits(bits, dev)
    st = torch.full((1,), scale, device=dev)
    amax = torch.zeros(1, device=dev)
    qb, q, sb, s = guarded_pair(*bits.shape, R.NVFP4, dev)
    fp8q.fp8q_fp4_quantize_amax(x, q, s, R.NVFP4, st, amax)
    check_packed(qb, q, sb, s, bits, R.NVFP4, scale)
    assert float(amax) == float("inf")
    tb, t, ub, u = guarded_pair(*bits.shape[::-1], R.NVFP4, dev)
    q2, s2 = torch.full_like(q, 0xEE), torch.full_like(s, 0xEE)
    fp8q.fp8q_fp4_quantize_amax(x, q2, s2, R.NVFP4, st, qt=t, sft=u)
    check_packed(tb, t, ub, u, np.ascontiguousarray(bits.T), R.NVFP4, scale)
    codes = slice(None)
    if R.quantize(bits, R.NVFP4, scale)[2].any():  # codes of a block whose scale is NaN are free
        codes = slice(0, 0)
    assert torch.equal(q2[codes], q[codes]) and torch.equal(s2, s)
    t2, u2 = torch.full_like(t, 0xEE), torch.full_like(u, 0xEE)
    fp8q.fp8q_fp4_quantize_amax(x, None, None, R.NVFP4, st, qt=t2, sft=u2)
    assert torch.equal(t2[codes], t[codes]) and torch.equal(u2, u)


@pytest.mark.parametrize("H", [64, 2064, 4096, 8208])
@pytest.mark.parametrize("scale", EDGES + OTHER + [1 / 3])
def test_norm_to_four_bits(dev, H, scale):
    """The codes are those of the h that the norm returns, whatever the scale; h is spread over many binades by the weight."""
    g = torch.Generator(device=dev)
    g.manual_seed(H)
    f = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    rows = 33
    x, block, post = f(rows, H).bfloat16(), f(rows, H).bfloat16(), 1 + 0.1 * f(H)
    pre = f(H) * torch.exp2(torch.randint(-60, 60, (H,), generator=g, device=dev).float()) * (scale if 0 < scale < 1e30 else 1.0)
    h, ro = torch.empty_like(x), torch.empty_like(x)
    st = torch.full((1,), scale, device=dev)
    qb, q, sb, s = guarded_pair(rows, H, R.NVFP4, dev)
    fp8q.fp8q_residual_norm_quantize_amax(x, ro, block=block, post_weight=post, pre_weight=pre, h=h, q=q, sf=s, fmt=R.NVFP4, scale=st)
    check_packed(qb, q, sb, s, bf16_bits_of(h).reshape(rows, H), R.NVFP4, scale)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("H", [64, 2064, 4096, 8208])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -126, 1e-40, 2.0 ** 100, 3e38, 0.0, -0.5, float("inf"), float("nan"), 1 / 3])
def test_norm_to_eight_bits(dev, H, scale, fmt):
    g = torch.Generator(device=dev)
    g.manual_seed(H)
    f = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    rows = 33
    x, block, post = f(rows, H).bfloat16(), f(rows, H).bfloat16(), 1 + 0.1 * f(H)
    pre = f(H) * torch.exp2(torch.randint(-20, 20, (H,), generator=g, device=dev).float()) * (scale if 0 < scale < 1e30 else 1.0)
    h, ro, q = torch.empty_like(x), torch.empty_like(x), torch.empty((rows, H), dtype=torch.uint8, device=dev)
    st = torch.full((1,), scale, device=dev)
    fp8q.fp8q_residual_norm_quantize_amax(x, ro, block=block, post_weight=post, pre_weight=pre, h=h, q=q, fmt=fmt, scale=st)
    want, _ = oracle.quantize_amax(bf16_bits_of(h), fmt, np.float32(scale))
    assert_codes_equal(q.cpu().numpy(), want, fmt)
