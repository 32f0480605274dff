"""Sums over a k that goes by parts: exact where no order can round them, close where it can, with the whole epilogue behind
them, and with waits that run out among the parts."""
import ctypes

import pytest
import torch

import fp8_reference as R
import test_gpu_fp8_give_up as give_up
import test_gpu_fp8_matmul as matmul
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_give_up import hooked  # noqa: F401
from test_gpu_fp8_grouped import experts
from test_gpu_fp8_matmul import gen, stored
from test_gpu_fp8_sums import small

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


# one more step than goes in one part, parts that end with a part of a step, an even and an odd number of parts; single CTAs (of
# 16 to 128 rows, k shared by clusters or not) and pairs, with vectors and without.  Sums of 140000 products of up to 16 in
# multiples of 1/4 stay below 2^24 of them, which binary32 holds in any order.
SHAPES = [(1, 640, 140000), (24, 19600, 16400), (40, 9800, 33001), (60, 9800, 40000), (128, 9800, 24600), (130, 9800, 40000), (300, 520, 130000),
          (2560, 2304, 16400), (2560, 2304, 33000), (2600, 2310, 24700), (300, 20016, 40970)]


@pytest.mark.parametrize("ta,tb", [(0, 0), (1, 1)])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_sums_that_cannot_round(dev, m, n, k, ta, tb):
    g = gen(dev, m + n + k)
    a, b = small((m, k), 0, g), small((n, k), 1, g)
    d = torch.empty((m, n), device=dev)
    fp8q.fp8q_matmul(stored(a, ta), stored(b, tb), d, 0, 1, a_trans=ta, b_trans=tb)
    want = sum(R.values(a[:, i: i + 8192], 0) @ R.values(b[:, i: i + 8192], 1).t() for i in range(0, k, 8192))
    assert torch.equal(d.double(), want)


@pytest.mark.parametrize("m,n", [(208, 528), (640, 130)])
@pytest.mark.parametrize("off", [[0, 16384, 16384, 33000, 33007, 90000], [5, 40000], [0, 100, 24577, 24600]])
def test_weight_gradients_that_cannot_round(dev, off, m, n):
    """Groups that go by parts beside others that do not, with and without what is there."""
    g = gen(dev, m + n)
    rows = off[-1] + 5
    a, b, at = small((rows, m), 1, g), small((rows, n), 0, g), torch.tensor(off, dtype=torch.int32, device=dev)
    d, old = torch.empty((len(off) - 1, m, n), device=dev), small((len(off) - 1, m, n), 0, g).view(torch.float8_e4m3fn).float()
    on_top = old.clone()
    fp8q.fp8q_grouped_weight_gradient(stored(a, 0), stored(b, 0), at, d)
    fp8q.fp8q_grouped_weight_gradient(stored(a, 0), stored(b, 0), at, on_top, residual=on_top)
    for i, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        want = R.values(a[lo:hi], 1).t() @ R.values(b[lo:hi], 0)
        assert torch.equal(d[i].double(), want) and torch.equal(on_top[i].double(), want + old[i].double())


@pytest.mark.parametrize("off", [[0, 2, 2, 30, 48], [0, 700, 1500, 1501, 3000]])
def test_rows_by_expert_that_cannot_round(dev, off):
    g = gen(dev, len(off))
    k, n = 33000, 1040
    a, (w, wt) = small((off[-1], k), 0, g), experts(4, n, k, 0, g)
    w[:] = small(w.shape, 0, g)
    wt.copy_(w)
    y = torch.empty((off[-1], n), device=dev)
    fp8q.fp8q_grouped_matmul(stored(a, 0), wt, torch.tensor(off, dtype=torch.int32, device=dev), y)
    for i, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        assert torch.equal(y[lo:hi].double(), R.values(a[lo:hi], 0) @ R.values(w[i], 0).t())


def off_by(got, want):
    return float(((got.double() - want).square().mean() / want.square().mean()).sqrt())


def test_errors_do_not_grow_with_k(dev):
    """A part's 256 multiply-adds of 32 cut off a step of binary32, 2^-23 of what they hold, at most, and each of the parts'
    additions rounds by half of one: of the results' root mean square (sums hold less on the way in the mean) 256 2^-23 for
    the parts together, whose errors and sums grow alike, and 2^-24 for each addition.  A million rows in one part were
    off by 3e-4."""
    g = gen(dev, 1)
    rows, n = 1 << 20, 256
    a, b = R.random_codes((rows, n), 0, g), R.random_codes((rows, n), 0, g)
    d = torch.empty((1, n, n), device=dev)
    fp8q.fp8q_grouped_weight_gradient(a, b, torch.tensor([0, rows], dtype=torch.int32, device=dev), d, 0, 0)
    want = sum(R.values(a[i: i + 65536], 0).t() @ R.values(b[i: i + 65536], 0) for i in range(0, rows, 65536))
    assert off_by(d[0], want) <= 256 * 2.0 ** -23 + rows / 8192 * 2.0 ** -24
    m, k = 300, 262144
    a, b = R.random_codes((m, k), 0, g), R.random_codes((520, k), 0, g)
    d = torch.empty((m, 520), device=dev)
    fp8q.fp8q_matmul(a, b, d)
    want = sum(R.values(a[:, i: i + 65536], 0) @ R.values(b[:, i: i + 65536], 0).t() for i in range(0, k, 65536))
    assert off_by(d, want) <= 256 * 2.0 ** -23 + k / 8192 * 2.0 ** -24


@pytest.mark.parametrize("m,n,k", [(24, 200, 140000), (130, 260, 66000), (2600, 2304, 16400), (2600, 2310, 24700)])
def test_the_epilogue_behind_parts(dev, m, n, k):
    """What holds of the epilogue at a short k, at this one."""
    matmul.test_codes_amax_and_checkpoint(dev, m, n, k, 0, 0.011)
    matmul.test_bias_gelu_residual(dev, m, n, k, torch.bfloat16)


@pytest.mark.parametrize("m,n", [(2600, 2320), (257, 20016)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_residual_over_many_tiles(dev, m, n, out):
    matmul.test_residual_over_many_tiles(dev, m, n, 16500, out, 16)


SUM_DRAINED = give_up.SUM_DRAINED


@pytest.mark.parametrize("role,at", [(give_up.COPY_EMPTY, 90), (give_up.SUM_FULL, 70), (SUM_DRAINED, 2), (give_up.OUT_DONE, 0)])
@pytest.mark.parametrize("m,n", [(40, 19600), (128, 9800)])
def test_waits_that_run_out_single_ctas(hooked, m, n, role, at):  # noqa: F811
    for dtype, cta in ((torch.bfloat16, -1), (torch.float32, 1)):
        f, want, got = give_up.product(m, n, 33024, dtype)
        assert give_up.check(hooked, f, want, got, role, at, cta).any()


@pytest.mark.parametrize("role,at", [(give_up.COPY_EMPTY, 200), (give_up.SUM_FULL, 70), (SUM_DRAINED, 2), (SUM_DRAINED, 5), (give_up.OUT_DONE, 2), (give_up.OUT_DONE, 5)])
def test_waits_that_run_out_pairs(hooked, role, at):  # noqa: F811
    """Tiles of three parts, so the first tile's result is the third set, the second's the sixth."""
    for dtype, cta in ((torch.bfloat16, -1), (torch.float32, 0)):
        f, want, got = give_up.product(4400, 2304, 16640, dtype)
        assert give_up.check(hooked, f, want, got, role, at, cta).any()


@pytest.mark.parametrize("role,at", [(give_up.MASK_FULL, 0), (give_up.SUM_DRAINED, 2), (give_up.SUM_FULL, 150)])
def test_waits_that_run_out_weight_gradients(hooked, role, at):  # noqa: F811
    dev = torch.device("cuda:0")
    g = gen(dev, 2)
    rows = 40000
    a, b = R.random_codes((rows, 528), 0, g), R.random_codes((rows, 304), 0, g)
    off = torch.tensor([0, 20001, 20001, rows], dtype=torch.int32, device=dev)
    want = torch.empty((3, 528, 304), device=dev)
    fp8q.fp8q_grouped_weight_gradient(a, b, off, want, 0, 0)
    got = torch.zeros_like(want)
    p = fp8q.Product(m=528, n=304, k=rows, a=a.data_ptr(), b=b.data_ptr(), lda=528, ldb=304, a_trans=1, b_trans=1, d=got.data_ptr(), out=1)
    f = lambda lib: lib.fp8q_grouped_weight_gradient(ctypes.byref(p), off.data_ptr(), 3, torch.cuda.current_stream().cuda_stream)  # noqa: E731
    for cta in (-1, 0):
        assert give_up.check(hooked, f, want, got, role, at, cta).any()
