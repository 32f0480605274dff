"""The products grouped by expert where offsets decrease: a row that one group holds has that group's result, one that several
hold has one of theirs, and a row of none is left as it was."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_grouped import experts
from test_gpu_fp8_matmul import gen, guarded, whole

pytestmark = pytest.mark.gpu


def spans(off, rows):
    """Each group's rows; bounds outside count as the nearest inside."""
    cut = [max(0, min(o, rows)) for o in off]
    return [range(lo, max(lo, hi)) for lo, hi in zip(cut[:-1], cut[1:])]


def drawn(rows, groups, seed):
    return torch.randint(-rows // 4, rows + rows // 4, (groups + 1,), generator=gen("cpu", seed)).tolist()


# few rows a group (single CTAs, whose grid has a part of a tile for each group) and many (pairs)
CASES = [(300, 200, [0, 200, 0, 200, 300]), (300, 130, [0, 150, 0, 300]), (300, 200, [0, 299, 0, 299, 0, 299, 0, 300]), (300, 200, [200, 300, 100, 150]),
         (60, 640, [10, 50, 0, 20, 60, 30]), (2000, 130, [0, 1990] * 20 + [2000, 1995]), (90, 130, [90, 0] * 30 + [90]),
         (3000, 1200, [0, 2000, 0, 2500, 3000]), (3000, 1200, [500, 2600, 0, 700, 3000])]
CASES += [(rows, n, drawn(rows, e, rows + e)) for rows, n, e in ((40, 130, 3), (200, 260, 9), (500, 130, 33), (777, 200, 65), (64, 130, 512), (4000, 1040, 7))]


@pytest.mark.parametrize("rows,n,off", CASES, ids=lambda v: str(v) if isinstance(v, int) else f"{len(v) - 1}groups")
def test_rows_of_offsets_that_decrease(rows, n, off):
    dev, k = torch.device("cuda:0"), 96
    g = gen(dev, rows + n)
    a, (w, wt) = R.random_codes((rows, k), 0, g), experts(len(off) - 1, n, k, 0, g)
    at = torch.tensor(off, dtype=torch.int32, device=dev)
    res = torch.randn((rows, n), generator=g, device=dev)
    held = torch.zeros(rows, dtype=torch.int32)
    for s in spans(off, rows):
        held[s.start: s.stop] += 1
    held = held.to(dev)
    assert (held > 0).any()
    for residual in (False, True):
        buf, d = guarded((rows, n), torch.float32, dev)
        d.fill_(77.0)
        fp8q.fp8q_grouped_matmul(a, wt, at, d, residual=res if residual else None)
        whole(buf)
        right = torch.zeros((rows, n), dtype=torch.bool, device=dev)
        for i, s in enumerate(spans(off, rows)):
            va, vb = R.values(a[s.start: s.stop], 0), R.values(w[i], 0)
            want = va @ vb.t() + (res[s.start: s.stop].double() if residual else 0.0)
            right[s.start: s.stop] |= (d[s.start: s.stop].double() - want).abs() <= R.sum_bound(va, vb) + 2.0 ** -23 * want.abs()
        assert right[held > 0].all(), "a row of a group that is not its product"
        assert (d[held == 0] == 77.0).all(), "a row of no group was written"
