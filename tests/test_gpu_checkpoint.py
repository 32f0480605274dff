"""The 8-bit checkpoint and the backward pass from it on the GPU: codes, scales and values bit for bit against the
definition in float64, gradients against float64 and against differences, sums over rows against float64."""
import numpy as np
import pytest
import torch

import fp8_reference as R
from gpu_helpers import bf16_bits_of
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp4 import from_bits, inputs
from test_gpu_fp8_matmul import gen, guarded, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (3, 64), (5, 96), (7, 4096), (129, 127), (130, 256), (1000, 48), (31, 2731), (257, 544), (9, 16384)]


def check_checkpoint(dev, bits, x):
    r, c = bits.shape
    codes, sf, val, nan = R.checkpoint(bits)
    bq, q = guarded((r, c), torch.uint8, dev)
    bs, s = guarded((r, (c + 31) // 32), torch.uint8, dev)
    fp8q.fp8q_checkpoint_quantize(x, q, s)
    whole(bq), whole(bs)
    assert np.array_equal(s.cpu().numpy(), sf), "scales differ"
    assert np.array_equal(q.cpu().numpy()[~nan], codes[~nan]), "codes differ"
    by, y = guarded((r, c), torch.bfloat16, dev)
    fp8q.fp8q_checkpoint_dequantize(q, s, y)
    whole(by)
    want = torch.from_numpy(val).to(dev).to(torch.float32).to(torch.bfloat16)  # exact in binary32
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y[~want.isnan()], want[~want.isnan()])
    fin = np.isfinite((bits.astype(np.uint32) << 16).view(np.float32)) & ~nan & np.isfinite(val)
    xv = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    step = np.repeat(np.exp2(sf.astype(np.float64) - 127 - 10), 32, 1)[:, :c]
    assert (np.abs(val[fin] - xv[fin]) <= np.maximum(np.abs(xv) / 16, step)[fin]).all()
    return q, s, val


@pytest.mark.parametrize("specials", [False, True])
@pytest.mark.parametrize("r,c", SHAPES)
def test_there_and_back(dev, r, c, specials):
    bits = inputs(r, c, r + c, specials)
    check_checkpoint(dev, bits, from_bits(bits, dev))


@pytest.mark.parametrize("off", [1, 8, 16])
@pytest.mark.parametrize("r,c", [(70, 96), (70, 100)])
def test_from_any_address(dev, r, c, off):
    bits = inputs(r, c, 5)
    room = torch.zeros(r * c + 64, dtype=torch.bfloat16, device=dev)
    x = room[off: off + r * c].view(r, c)
    x.copy_(from_bits(bits, dev))
    check_checkpoint(dev, bits, x)


@pytest.mark.parametrize("cols", [32, 31])
def test_every_bf16_alone_and_beside_a_larger_one(dev, cols):
    """Every finite pattern as a block's largest, and (second column) within blocks of every scale."""
    p = np.arange(65536, dtype=np.uint16)
    bits = np.zeros((65536, cols), np.uint16)
    bits[:, 0] = p
    bits[:, 3] = p[::-1]
    check_checkpoint(dev, bits, from_bits(bits, dev))


def grad_inputs(dev, r, c, seed, spread=1.0):
    g = gen(dev, seed)
    h = (torch.randn((r, c), generator=g, device=dev) * spread).to(torch.bfloat16)
    dy = (torch.randn((r, c), generator=g, device=dev) * 1e-2).to(torch.bfloat16)
    q, sf = fp8q.checkpoint_empty(r, c)
    fp8q.fp8q_checkpoint_quantize(h, q, sf)
    v = torch.empty_like(h)
    fp8q.fp8q_checkpoint_dequantize(q, sf, v)
    return dy, q, sf, v.double()


def back(dev, dy, q, sf, fmt=1, scale=1e-3, bias=True, codes=True, dx=True):
    r, c = dy.shape
    out = {"d_x": guarded((r, c), torch.bfloat16, dev) if dx else (None, None), "q": guarded((r, c), torch.uint8, dev) if codes else (None, None),
           "d_bias": guarded((c,), torch.float32, dev) if bias else (None, None)}
    amax = torch.zeros(1, device=dev)
    space = torch.empty(fp8q.gelu_backward_workspace(r, c), dtype=torch.uint8, device=dev) if bias else None
    fp8q.fp8q_gelu_backward_quantize_amax(dy, q, sf, out["q"][1], fmt, torch.full((1,), scale, device=dev) if codes else None, amax,
                                          out["d_x"][1], out["d_bias"][1], space)
    for b, _ in out.values():
        if b is not None:
            whole(b)
    return {k: t for k, (_, t) in out.items()} | {"amax": amax}


@pytest.mark.parametrize("spread", [0.1, 1.0, 6.0, 1e4])
@pytest.mark.parametrize("gelu", [True, False])
@pytest.mark.parametrize("r,c", [(1, 1), (1, 8), (3, 33), (33, 40), (64, 256), (130, 257), (777, 1552), (1000, 2731), (20000, 3)])
def test_gelu_backward(dev, r, c, gelu, spread):
    dy, q, sf, v = grad_inputs(dev, r, c, r + c, spread)
    if not gelu:
        q = sf = None
    got = back(dev, dy, q, sf)
    slope = R.gelu_slope(v) if gelu else torch.ones_like(v)
    want = dy.double() * slope
    # the slope, the product and the rounding to bf16
    off = dy.double().abs() * (2.0 ** -19 * (1 + v.abs().clamp(max=10))) * (1 if gelu else 0) + 2.0 ** -24 * want.abs()
    assert ((got["d_x"].double() - want).abs() <= off + 2.0 ** -8 * (want.abs() + off) + 2.0 ** -134).all()
    # codes and amax: those of d_x
    q2, a2 = torch.empty((r, c), dtype=torch.uint8, device=dev), torch.zeros(1, device=dev)
    fp8q.fp8q_quantize_amax(got["d_x"], q2, 1, torch.full((1,), 1e-3, device=dev), a2)
    assert torch.equal(got["q"], q2) and torch.equal(got["amax"], a2)
    # the sums: each term as above, and a rounding for each row
    bound = off.sum(0) + (r + 2) * 2.0 ** -24 * want.abs().sum(0)
    assert ((got["d_bias"].double() - want.sum(0)).abs() <= bound).all()
    # parts alone give the same bits
    for parts in (dict(bias=False), dict(codes=False), dict(dx=False), dict(codes=False, dx=False), dict(bias=False, dx=False, fmt=1)):
        one = back(dev, dy, q, sf, **parts)
        assert all(torch.equal(one[k], got[k]) for k in one if one[k] is not None)
    e4 = back(dev, dy, q, sf, fmt=0, scale=2.0 ** -65)["q"]
    fp8q.fp8q_quantize_amax(got["d_x"], q2, 0, torch.full((1,), 2.0 ** -65, device=dev), a2)
    assert torch.equal(e4, q2)


def test_slope_against_differences(dev):
    """The derivative against central differences of the GELU in 64 bits, at every value a checkpoint of one scale holds."""
    codes = torch.arange(256, dtype=torch.uint8, device=dev)
    codes[[0x7F, 0xFF]] = 0
    q = codes.view(1, 256).repeat(24, 1)
    sf = torch.arange(127 - 18, 127 + 6, dtype=torch.uint8, device=dev)[:, None].repeat(1, 8)
    dy = torch.ones((24, 256), dtype=torch.bfloat16, device=dev)
    d_bias = torch.empty(256, device=dev)
    for i in range(24):  # a row at a time: d_bias is the slope, unrounded
        fp8q.fp8q_gelu_backward_quantize_amax(dy[i: i + 1], q[i: i + 1], sf[i: i + 1], d_bias=d_bias)
        x = R.values(q[i], 0) * 2.0 ** (float(sf[i, 0]) - 127)
        near = x.abs() < 12
        step = 1e-5 * (1 + x.abs())
        diff = (R.gelu(x + step) - R.gelu(x - step)) / (2 * step)
        # differences are off by step^2 / 6 of the third derivative (under 3) and by 2^-52 |gelu| / step
        assert ((d_bias.double() - diff).abs() <= 2.0 ** -19 * (1 + x.abs()) + step ** 2 + 2.0 ** -50 * (1 + x.abs()) / step)[near].all()
        assert (d_bias[~near] == (x[~near] > 0).float()).all()


def test_gelu_backward_specials(dev):
    x = torch.tensor([[float("inf"), -float("inf"), 3e38, -3e38, 0.0, -0.0, 1e-40, 2.0] * 4, [float("nan")] + [1.0] * 31], device=dev).to(torch.bfloat16)
    q, sf = fp8q.checkpoint_empty(2, 32)
    fp8q.fp8q_checkpoint_quantize(x, q, sf)
    dy = torch.full((2, 32), 0.5, dtype=torch.bfloat16, device=dev)
    got = back(dev, dy, q, sf)
    assert torch.equal(got["d_x"][0, :6].float(), torch.tensor([0.5, 0, 0.5, 0, 0.25, 0.25], device=dev))
    assert torch.isnan(got["d_x"][1]).all() and torch.isnan(got["amax"]).all() and torch.isnan(got["d_bias"]).all()
    dy[0, 0], dy[0, 2] = float("nan"), float("inf")
    d = back(dev, dy[:1], q[:1], sf[:1])["d_x"]
    assert torch.isnan(d[0, 0]) and d[0, 2] == float("inf") and torch.isfinite(d[0, 3:]).all()


def test_no_rows_and_workspace(dev):
    none = torch.empty((0, 40), dtype=torch.bfloat16, device=dev)
    d = torch.ones(40, device=dev)
    fp8q.fp8q_gelu_backward_quantize_amax(none, None, None, d_bias=d)
    assert not d.any()
    dy = torch.ones((4000, 40), dtype=torch.bfloat16, device=dev)
    need = fp8q.gelu_backward_workspace(4000, 40)
    assert need > 0 and need % 160 == 0
    with pytest.raises(fp8q.Fp8qError):
        fp8q.fp8q_gelu_backward_quantize_amax(dy, None, None, d_bias=d, workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev))
    buf = torch.full((need + 512,), 0xEE, dtype=torch.uint8, device=dev)
    fp8q.fp8q_gelu_backward_quantize_amax(dy, None, None, d_bias=d, workspace=buf[256: 256 + need])
    assert (d == 4000).all() and (buf[:256] == 0xEE).all() and (buf[256 + need:] == 0xEE).all()


def test_refusals(dev):
    dy = torch.ones((4, 40), dtype=torch.bfloat16, device=dev)
    h, sf = fp8q.checkpoint_empty(4, 40)
    d, one = torch.empty(40, device=dev), torch.ones(1, device=dev)
    for bad in (dict(h=h[:3]), dict(h_sf=sf[:, :1].contiguous()), dict(d_bias=d[:39]), dict(d_y=dy.float()), dict(d_y=dy.t()), dict(scale=torch.ones(2, device=dev)),
                dict(d_y=dy.cpu()), dict(q=h[:3])):
        with pytest.raises(ValueError):
            fp8q.fp8q_gelu_backward_quantize_amax(**{**dict(d_y=dy, h=h, h_sf=sf, d_bias=d), **bad})
    for bad in (dict(d_bias=None), dict(h=None), dict(q=h), dict(scale=one), dict(fmt=2)):
        with pytest.raises(fp8q.Fp8qError):
            fp8q.fp8q_gelu_backward_quantize_amax(**{**dict(d_y=dy, h=h, h_sf=sf, d_bias=d), **bad})
    with pytest.raises(ValueError):
        fp8q.fp8q_checkpoint_quantize(dy, h, sf[:3])
    with pytest.raises(ValueError):
        fp8q.fp8q_checkpoint_dequantize(h, sf, dy[:3])


@pytest.mark.parametrize("cols", [1, 7, 8, 9, 40, 248, 255, 256, 257, 263, 265, 511, 784, 2047, 2049, 4101])
def test_rows_and_outputs_from_any_address(dev, cols):
    """Inputs and outputs at every offset from the vectors that hold them, rows of every length beside 256."""
    for rows, x_off, q_off, y_off in ((1, 0, 0, 0), (3, 1, 1, 1), (5, 7, 7, 7), (4, 3, 2, 6), (9, 8, 3, 2), (2, 5, 4, 5), (40, 2, 5, 3), (33, 6, 6, 4), (7, 16, 0, 16), (70, 16, 16, 0)):
        bits = inputs(rows, cols, rows + cols, rows % 2 == 0)
        codes, sf, val, nan = R.checkpoint(bits)
        n, blocks = rows * cols, (cols + 31) // 32
        x = torch.zeros(x_off + n, dtype=torch.bfloat16, device=dev)[x_off:].view(rows, cols)
        x.copy_(from_bits(bits, dev))
        bq = torch.full((n + 64,), 0xEE, dtype=torch.uint8, device=dev)
        bs = torch.full((rows * blocks + 64,), 0xEE, dtype=torch.uint8, device=dev)
        by = torch.full((n + 64,), -7.0, dtype=torch.bfloat16, device=dev)
        q, s = bq[16 + q_off: 16 + q_off + n].view(rows, cols), bs[16 + q_off: 16 + q_off + rows * blocks].view(rows, blocks)
        y = by[16 + y_off: 16 + y_off + n].view(rows, cols)
        fp8q.fp8q_checkpoint_quantize(x, q, s)
        fp8q.fp8q_checkpoint_dequantize(q, s, y)
        for buf, off, size, old in ((bq, 16 + q_off, n, 0xEE), (bs, 16 + q_off, rows * blocks, 0xEE), (by, 16 + y_off, n, -7.0)):
            assert (buf[:off] == old).all() and (buf[off + size:] == old).all(), "write outside the output"
        assert np.array_equal(s.cpu().numpy(), sf), "scales differ"
        assert np.array_equal(q.cpu().numpy()[~nan], codes[~nan]), "codes differ"
        want = torch.from_numpy(val).to(dev).to(torch.float32).to(torch.bfloat16)
        assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y[~want.isnan()], want[~want.isnan()])
