"""Waits of the 4-bit product that run out, without any fault.

Every wait of the product's kernels is bounded; one that runs out shows as NaN, all the bits behind the sign set, where
the product is not what it should be.  In correct operation none does, so these tests use the library built once more
with its test hooks: one wait, of one role at one step, reports failure in a single lane of its warp although what it
waits for has come.  The warp has to take it as one verdict (lanes that parted would never meet again at the warp-wide
instructions that follow), the warps that wait for it have to run out in their turn (after a tenth of a second in that
build), and the call has to end, with NaN or the right value in every element and the device as usable as before."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_reference as R
from quantize_amax_scaling_gb300 import fp8q

pytestmark = pytest.mark.gpu

COPY_EMPTY, SUM_FULL, SUM_SCALED, SCALE_FULL, OUT_DONE, SCALE_COPY_EMPTY, SUM_DRAINED = range(1, 8)


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


@pytest.fixture
def hooked(hooks_lib):
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    hooks_lib.fp8q_fp4_matmul.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, vp, vp]
    hooks_lib.fp8q_test_set_matmul_give_up.argtypes = [i32, i32, i32]
    hooks_lib.fp8q_test_set_matmul_give_up.restype = None
    yield hooks_lib
    hooks_lib.fp8q_test_set_matmul_give_up(0, 0, -1)


def operand(r, c, fmt, seed, dev):
    rng = np.random.RandomState(seed)
    q, s = R.pack(rng.randint(0, 16, (r, c)).astype(np.uint8),
                  rng.randint(*((120, 134) if fmt == R.MXFP4 else (0x20, 0x50)), (r, -(-c // R.BLOCK[fmt]))).astype(np.uint8))
    return torch.from_numpy(q).to(dev), torch.from_numpy(s).to(dev)


def check(hooked, dev, m, n, k, fmt, dtype, role, at, cta):
    a, b = operand(m, k, fmt, 1, dev), operand(n, k, fmt, 2, dev)
    want = torch.empty((m, n), dtype=dtype, device=dev)
    fp8q.fp8q_fp4_matmul(*a, *b, want, k, fmt)
    got = torch.zeros_like(want)

    def call():
        assert hooked.fp8q_fp4_matmul(*(t.data_ptr() for t in (*a, *b, got)), m, n, k, fmt, int(dtype == torch.float32), None, None,
                                      torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()  # the call ends: nothing waits forever

    hooked.fp8q_test_set_matmul_give_up(role, at, cta)
    call()
    ints, top = (torch.int32, 0x7FFFFFFF) if dtype == torch.float32 else (torch.int16, 0x7FFF)
    lost = (got.view(ints) & top) == top
    assert torch.equal(got[~lost], want[~lost]), "an element that is neither right nor NaN"
    hooked.fp8q_test_set_matmul_give_up(0, 0, -1)
    got.zero_()
    call()
    assert torch.equal(got, want), "the same kernel behind one that gave up"
    return lost


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("role,at", [(COPY_EMPTY, 0), (COPY_EMPTY, 1), (SUM_FULL, 0), (SUM_FULL, 1), (SUM_SCALED, 1), (SCALE_FULL, 0),
                                     (SCALE_FULL, 1), (OUT_DONE, 0)])
@pytest.mark.parametrize("m,n,k", [(1, 640, 4096), (40, 256, 8192), (65, 200, 1033), (300, 520, 320)])
def test_single_ctas(hooked, dev, m, n, k, role, at, fmt):
    """Clusters of CTAs that share sums, and CTAs by themselves."""
    assert check(hooked, dev, m, n, k, fmt, torch.bfloat16, role, at, -1).all()
    lost = check(hooked, dev, m, n, k, fmt, torch.float32, role, at, 1)  # one CTA of them: its tile
    assert lost.any() and int(lost.sum()) <= 128 * 128


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("role,at", [(COPY_EMPTY, 0), (COPY_EMPTY, 7), (SCALE_COPY_EMPTY, 0), (SCALE_COPY_EMPTY, 3), (SUM_FULL, 0), (SUM_FULL, 1),
                                     (SUM_FULL, 6), (SUM_FULL, 9), (SCALE_FULL, 0), (SCALE_FULL, 5), (SUM_DRAINED, 1), (OUT_DONE, 0),
                                     (OUT_DONE, 1)])
@pytest.mark.parametrize("m,n,k", [(2560, 2304, 1100), (2700, 2751, 1100)])
def test_pairs(hooked, dev, m, n, k, role, at, fmt):
    """Pairs of CTAs, the first of which take two tiles of 256 x 256, 5 steps each: what a pair had not
    finished when it gave up is NaN, also where sums of a part of k were there."""
    for dtype, cta in ((torch.bfloat16, -1), (torch.float32, 0), (torch.bfloat16, 1)):
        if cta == 1 and role in (SUM_FULL, SUM_DRAINED):
            continue  # the first CTA of a pair issues for both
        lost = check(hooked, dev, m, n, k, fmt, dtype, role, at, cta)
        assert lost.any() and (cta < 0 or int(lost.sum()) <= 2 * 256 * 256)
        if role == SUM_FULL and cta == 0 and at < k // 256:  # in the pair's first tile
            assert lost[:256, :256].all()
