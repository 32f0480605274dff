"""The FP8 products' sums over a long k.  Small whole and half codes, whose sums no order and no alignment of the addends can
round: bit for bit the exact ones, so that no product is left out or counted twice.  And sums of ordinary codes, within what
the additions of k can cut off."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_grouped import experts
from test_gpu_fp8_matmul import gen, operands, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def small(shape, fmt, g):
    """Codes of 0, and of 0.5, 1, 1.5, 2, 3 and 4 with either sign.  Products are multiples of 2^-2 up to 2^4; a sum of 2^14 of them
    is below 2^18 and a multiple of 2^-2, in whatever order: 20 bits, and binary32 holds 24."""
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, -0.5, -1, -1.5, -2, -3, -4], device=g.device)
    return v[torch.randint(0, 13, shape, generator=g, device=g.device)].to(R.DTYPE[fmt]).view(torch.uint8)


# one token and few (clusters of 8 to 1), several tiles, pairs, and widths without vectors in both kernels
SHAPES = [(1, 640, 16384), (1, 16384, 4096), (24, 512, 16384), (65, 201, 8208), (127, 1040, 4100), (300, 520, 8192), (1003, 1040, 2064),
          (2560, 2304, 4096), (2600, 2320, 16384), (2600, 2310, 4096)]


@pytest.mark.parametrize("ta,tb", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_sums_that_cannot_round(dev, m, n, k, ta, tb):
    g = gen(dev, m + n + k)
    fa, fb = (m + ta) % 2, (n + tb) % 2
    a, b = small((m, k), fa, g), small((n, k), fb, g)
    d = torch.empty((m, n), device=dev)
    fp8q.fp8q_matmul(stored(a, ta), stored(b, tb), d, fa, fb, a_trans=ta, b_trans=tb)
    assert torch.equal(d.double(), R.values(a, fa) @ R.values(b, fb).t())


@pytest.mark.parametrize("off,m,n", [([0, 5000, 5000, 5033, 12000], 208, 528), ([3, 4100, 9000, 16387], 640, 130), ([0, 16384], 256, 256)])
def test_weight_gradients_that_cannot_round(dev, off, m, n):
    g = gen(dev, m + n)
    rows = off[-1] + 5
    a, b, at = small((rows, m), 1, g), small((rows, n), 0, g), torch.tensor(off, dtype=torch.int32, device=dev)
    d = torch.empty((len(off) - 1, m, n), device=dev)
    fp8q.fp8q_grouped_weight_gradient(stored(a, 0), stored(b, 0), at, d)
    for i, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        assert torch.equal(d[i].double(), R.values(a[lo:hi], 1).t() @ R.values(b[lo:hi], 0))


@pytest.mark.parametrize("off", [[0, 2, 2, 30, 48], [0, 700, 1500, 1501, 4000]])
def test_rows_by_expert_that_cannot_round(dev, off):
    g = gen(dev, len(off))
    k, n = 8192, 1040
    a, (w, wt) = small((off[-1], k), 0, g), experts(4, n, k, 0, g)
    w[:] = small(w.shape, 0, g)
    wt.copy_(w)
    y = torch.empty((off[-1], n), device=dev)
    fp8q.fp8q_grouped_matmul(a, wt, torch.tensor(off, dtype=torch.int32, device=dev), y)
    for i, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        assert torch.equal(y[lo:hi].double(), R.values(a[lo:hi], 0) @ R.values(w[i], 0).t())


@pytest.mark.parametrize("m,n,k", [(16, 2048, 16384), (300, 520, 8192), (2560, 2304, 4096), (2560, 2304, 16384)])
def test_what_a_long_k_cuts_off(dev, m, n, k):
    """Each of k / 32 multiply-adds cuts its sum off at a step of binary32 at most, 2^-23 of what it holds, which is no more than
    the result in the mean over the matrix (sums of products of either sign grow with the root of their number); what it cuts off of
    the products is below that step too, and of either sign.  So errors are within k / 32 2^-23 of the results in their root
    mean square: 1.5e-5 at 4096, where a product left out of each sum would be off by 1.6e-2."""
    a, b = operands(dev, m, n, k, 5)
    va, vb = R.values(a, 0), R.values(b, 0)
    d = torch.empty((m, n), device=dev)
    fp8q.fp8q_matmul(a, b, d)
    want = va @ vb.t()
    off = ((d.double() - want).square().mean() / want.square().mean()).sqrt()
    print(f"off by {float(off):.2g} of the root mean square")
    assert off <= k / 32 * 2.0 ** -23
