"""The FP8 products, checkpoints and gradients beyond 2^31 and 2^32 elements: offsets in 64 bits, on rows near both ends."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_matmul import check, gen

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("m,n", [(140000, 32000), (20, 230000000)])
def test_products(m, n):
    """Outputs of more than 2^32 elements, from pairs of CTAs and from single ones."""
    g = gen(DEV, 1)
    a, b = R.random_codes((m, 16), 0, g), R.random_codes((n, 16), 0, g)
    q = torch.empty((m, n), dtype=torch.uint8, device=DEV)
    one, amax = torch.ones(1, device=DEV), torch.zeros(1, device=DEV)
    d = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    fp8q.fp8q_matmul(a, b, d, q=q, q_scale=one, amax=amax)
    for r in (slice(0, 3), slice(m - 3, m)):
        for c in (slice(0, 300), slice(n - 300, n)):
            va, vb = R.values(a[r], 0), R.values(b[c].contiguous(), 0)
            check(d[r, c], va @ vb.t(), R.sum_bound(va, vb))
            want = torch.empty((3, 300), dtype=torch.uint8, device=DEV)
            fp8q.fp8q_quantize_amax(d[r, c].contiguous(), want, 0, one, torch.zeros(1, device=DEV))
            assert torch.equal(q[r, c], want)
    assert float(amax) == max(float(d[i: i + 20000].abs().max()) for i in range(0, m, 20000))


def test_grouped():
    """Weights and gradients of more than 2^32 elements in all groups."""
    e, n, k = 40, 8192, 16384
    g = gen(DEV, 2)
    w = R.random_codes((1, n, k), 0, g).expand(e, n, k).contiguous()
    w[-1] ^= 0x80
    x, off = R.random_codes((80, k), 0, g), torch.arange(0, 82, 2, dtype=torch.int32, device=DEV)
    y = torch.empty((80, n), device=DEV)
    fp8q.fp8q_grouped_matmul(x, w, off, y)
    v = R.values(w[0], 0)
    for r, s in ((slice(0, 2), 1), (slice(76, 78), 1), (slice(78, 80), -1)):
        va = R.values(x[r], 0)
        check(y[r], s * (va @ v.t()), R.sum_bound(va, v))
    del w
    d = torch.empty((e, n, k), dtype=torch.bfloat16, device=DEV)
    a = R.random_codes((80, n), 0, g)
    fp8q.fp8q_grouped_weight_gradient(a, x, off, d, 0, 0)
    for i in (0, e - 1):
        va, vb = R.values(a[2 * i: 2 * i + 2], 0).t(), R.values(x[2 * i: 2 * i + 2], 0).t()
        check(d[i], va @ vb.t(), R.sum_bound(va, vb))


@pytest.mark.parametrize("r,c", [(70000, 65536), (70000, 65537)])
def test_checkpoint_and_back(r, c):
    x = torch.empty((r, c), dtype=torch.bfloat16, device=DEV)
    for i in range(0, r, 10000):
        x[i: i + 10000] = torch.randn((min(10000, r - i), c), device=DEV)
    h, s = fp8q.checkpoint_empty(r, c)
    fp8q.fp8q_checkpoint_quantize(x, h, s)
    y, q, amax = torch.empty_like(x), torch.empty((r, c), dtype=torch.uint8, device=DEV), torch.zeros(1, device=DEV)
    fp8q.fp8q_checkpoint_dequantize(h, s, y)
    space, db, one = torch.empty(fp8q.gelu_backward_workspace(r, c), dtype=torch.uint8, device=DEV), torch.empty(c, device=DEV), torch.ones(1, device=DEV)
    fp8q.fp8q_gelu_backward_quantize_amax(x, h, s, q, 0, one, amax, d_bias=db, workspace=space)
    for rows in (slice(0, 5), slice(r - 5, r)):
        h2, s2 = fp8q.checkpoint_empty(5, c)
        fp8q.fp8q_checkpoint_quantize(x[rows].contiguous(), h2, s2)
        assert torch.equal(h2, h[rows]) and torch.equal(s2, s[rows])
        y2, q2 = torch.empty((5, c), dtype=torch.bfloat16, device=DEV), torch.empty((5, c), dtype=torch.uint8, device=DEV)
        fp8q.fp8q_checkpoint_dequantize(h2, s2, y2)
        fp8q.fp8q_gelu_backward_quantize_amax(x[rows].contiguous(), h2, s2, q2, 0, one)
        assert torch.equal(y2, y[rows]) and torch.equal(q2, q[rows])
    for col in (0, c - 40):
        t = x[:, col: col + 40].double() * R.gelu_slope(y[:, col: col + 40])
        bound = (r + 2) * 2.0 ** -24 * t.abs().sum(0) + 2.0 ** -19 * (x[:, col: col + 40].double().abs() * (1 + y[:, col: col + 40].double().abs())).sum(0)
        assert ((db[col: col + 40].double() - t.sum(0)).abs() <= bound).all()
