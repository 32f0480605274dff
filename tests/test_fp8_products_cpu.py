"""Refusals of the FP8 products, the checkpoint and the GELU's backward pass, through the C entry points: each comes back
before anything is launched, so none of this needs a GPU.  And the tests' reference against plain arithmetic."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import fp8_reference as R

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from quantize_amax_scaling_gb300 import build, fp8q
    build.build()
    return fp8q.lib()


def product(**over):
    from quantize_amax_scaling_gb300.fp8q import Product
    good = dict(m=8, n=16, k=32, a=P, b=P, lda=32, ldb=32, d=P, out=0)
    return Product(**{**good, **over})


def codes(L, name, *more, **over):
    p = product(**over)
    return getattr(L, name)(ctypes.byref(p), *more, None)


def test_matmul_refusals(L):
    f = lambda **o: codes(L, "fp8q_matmul", **o)  # noqa: E731
    assert L.fp8q_matmul(None, None) == INVALID
    for bad in (dict(m=-1), dict(n=-1), dict(k=-1), dict(a_fmt=2), dict(b_fmt=3), dict(out=2), dict(act=2), dict(a=None), dict(b=None), dict(d=None),
                dict(lda=31), dict(ldb=16), dict(q=P), dict(q_scale=P), dict(q=P, q_scale=P, q_fmt=2), dict(out=1, q=P, q_scale=P), dict(out=1, amax=P),
                dict(out=1, d=None, h=P, h_sf=P), dict(h=P), dict(h_sf=P), dict(d=P + 1), dict(out=1, d=P + 2), dict(residual=P + 1), dict(bias=P + 2),
                dict(bias=P + 1, bias_is_bf16=1), dict(a_scale=P + 2), dict(b_scale=P + 1), dict(q=P, q_scale=P + 2), dict(amax=P + 2),
                dict(a_trans=1, lda=0), dict(b_trans=1, ldb=0)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(a=P + 8), dict(b=P + 1), dict(lda=40), dict(ldb=33), dict(m=2 ** 31), dict(n=2 ** 31 - 1023), dict(k=2 ** 40, lda=2 ** 40, ldb=2 ** 40),
                dict(lda=2 ** 31), dict(ldb=2 ** 33)):
        assert f(**bad) == UNSUPPORTED, bad
    for empty in (dict(m=0), dict(n=0), dict(m=0, d=None, a=None)):
        assert f(**empty) == OK


def test_grouped_refusals(L):
    f = lambda off=P, g=3, **o: codes(L, "fp8q_grouped_matmul", off, g, **o)  # noqa: E731
    assert f(g=-1) == INVALID and f(off=None) == INVALID and f(off=P + 2) == INVALID and f(a_trans=1) == INVALID
    assert f(g=513) == UNSUPPORTED and f(a=P + 4) == UNSUPPORTED
    assert f(g=512, n=2 ** 30, ldb=1024) == UNSUPPORTED  # a matrix to the next: 2^40 bytes
    assert f(g=0) == OK and f(m=0) == OK and f(g=0, off=None) == OK
    h = lambda off=P, g=3, **o: codes(L, "fp8q_grouped_weight_gradient", off, g, **{**dict(a_trans=1, b_trans=1), **o})  # noqa: E731
    for bad in (dict(a_trans=0), dict(b_trans=0), dict(bias=P), dict(act=1), dict(q=P, q_scale=P), dict(amax=P), dict(h=P, h_sf=P), dict(off=None), dict(g=-1),
                dict(d=None), dict(lda=0)):
        assert h(**bad) == INVALID, bad
    assert h(g=513) == UNSUPPORTED and h(b=P + 2) == UNSUPPORTED
    assert h(g=0) == OK and h(n=0) == OK


def test_checkpoint_refusals(L):
    q, d = L.fp8q_checkpoint_quantize, L.fp8q_checkpoint_dequantize
    for f, x, rest in ((q, 0, (1, 2)), (d, 2, (0, 1))):
        good = [P, P, P, 4, 40, None]
        call = lambda i, v: f(*[v if j == i else a for j, a in enumerate(good)])  # noqa: E731
        for i in range(3):
            assert call(i, None) == INVALID
        assert call(x, P + 1) == INVALID and call(3, -1) == INVALID and call(4, -1) == INVALID
        assert call(3, 2 ** 31) == UNSUPPORTED and call(4, 2 ** 31 - 1023) == UNSUPPORTED
        assert f(None, None, None, 0, 40, None) == OK and f(None, None, None, 4, 0, None) == OK
    assert [L.fp8q_checkpoint_scale_bytes(*s) for s in ((3, 1), (3, 32), (3, 33), (0, 5), (-1, 5), (5, 2 ** 31))] == [3, 3, 6, 0, 0, 0]


def test_gelu_backward_refusals(L):
    from quantize_amax_scaling_gb300.fp8q import GeluGrad

    def f(**over):
        g = GeluGrad(**{**dict(rows=4, cols=40, fmt=1, d_y=P, h=P, h_sf=P, q=P, scale=P, d_x=P), **over})
        return L.fp8q_gelu_backward_quantize_amax(ctypes.byref(g), None)

    assert L.fp8q_gelu_backward_quantize_amax(None, None) == INVALID
    for bad in (dict(rows=-1), dict(cols=-1), dict(fmt=2), dict(d_y=None), dict(h=None), dict(h_sf=None), dict(q=None), dict(scale=None),
                dict(q=None, scale=None, d_x=None), dict(d_y=P + 1), dict(d_x=P + 1), dict(scale=P + 2), dict(amax=P + 1), dict(d_bias=P + 2),
                dict(rows=4000, d_bias=P), dict(rows=4000, d_bias=P, workspace=P, workspace_bytes=100),
                dict(rows=4000, d_bias=P, workspace=P + 2, workspace_bytes=1 << 20)):
        assert f(**bad) == INVALID, bad
    assert f(rows=2 ** 31) == UNSUPPORTED and f(cols=2 ** 31) == UNSUPPORTED
    assert f(cols=0) == OK and f(rows=0) == OK
    w = L.fp8q_gelu_backward_workspace
    assert w(0, 5) == w(5, 0) == w(-1, 5) == w(2 ** 31, 5) == 0 and w(1, 4096) == 0
    assert 0 < w(8192, 16384) <= 64 * 16384 * 4


def test_reference_checkpoint_by_fractions():
    """The reference's scales and codes against a search over all of them in exact arithmetic."""
    rng = np.random.RandomState(4)
    bits = rng.randint(0, 0x7F80, (12, 40)).astype(np.uint16) | (rng.randint(0, 2, (12, 40)).astype(np.uint16) << 15)
    bits[3] = rng.randint(0x3F00, 0x4100, 40)
    bits[4, 5] = 0x7F80
    bits[5, 33] = 0x7FC1
    bits[6] = 0
    codes, sf, val, nan = R.checkpoint(bits)
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    table = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    top = Fraction(float(np.uint32(0x7F7F0000).view(np.float32)))
    for r in range(12):
        for b in range(2):
            blk = x[r, 32 * b: 32 * b + 32]
            if np.isnan(blk).any():
                assert sf[r, b] == 255 and nan[r, 32 * b]
                continue
            a = max(min(abs(Fraction(float(v))), top) if np.isfinite(v) else top for v in blk)
            e = next(i for i in range(-127, 128) if a <= 448 * Fraction(2) ** i)
            assert sf[r, b] == e + 127
            for j, v in enumerate(blk):
                m = min(abs(Fraction(float(v))) / Fraction(2) ** e, Fraction(448)) if np.isfinite(v) else Fraction(448)
                d = [abs(Fraction(float(t)) - m) for t in table]
                near = [i for i in range(127) if d[i] == min(d)]
                c = near[0] if len(near) == 1 else next(i for i in near if i % 2 == 0)
                assert codes[r, 32 * b + j] == c | (0x80 if np.signbit(v) else 0)


def test_reference_slope_by_differences():
    x = torch.linspace(-12, 12, 2001, dtype=torch.float64)
    h = 1e-5
    assert ((R.gelu(x + h) - R.gelu(x - h)) / (2 * h) - R.gelu_slope(x)).abs().max() < 1e-9
