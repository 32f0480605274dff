"""The residual norms' rows whose mean of squares is no finite number: NaN in every column, nothing in other rows."""
import pytest
import torch

import fp4_reference as R
from test_gpu_residual_norm import forward, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


# 3e19 squared is 9e38, beyond binary32's 3.4e38; 1e19 squared is 1e38, and two or three of them are within it
TOO_LARGE = [("nan", 1), ("inf", 1), ("-inf", 1), (3e19, 1), (3.3e38, 1), (1e19, 5), (1.5e18, 10 ** 9)]


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
@pytest.mark.parametrize("H", [64, 1040, 2064, 4096, 8208, 16384])
@pytest.mark.parametrize("value,times", TOO_LARGE)
def test_rows_that_no_mean_holds(dev, H, fmt, value, times):
    if value == 1.5e18 and H < 256:
        pytest.skip("64 squares of 2.25e36 are within binary32")
    rows = 12
    clean = make(rows, H, 5, "f32", H, dev)
    want = forward(clean, rows, H, 5, 0.5, 1e-6, fmt=fmt, dev=dev)
    for where in ("block", "residual"):
        d = dict(clean, **{where: clean[where].clone()})
        for row in (0, 4, 11):
            d[where][row, row: row + times] = float(value)
        o = forward(d, rows, H, 5, 0.5, 1e-6, fmt=fmt, dev=dev)
        for row in range(rows):
            if row not in (0, 4, 11):
                assert all(torch.equal(o[k][row], want[k][row]) for k in ("ro", "h", "rstd_pre", "rstd_post")), (where, row)
                continue
            assert torch.isnan(o["h"][row]).all() and torch.isnan(o["rstd_pre"][row]), (where, row)
            if where == "block":
                assert torch.isnan(o["ro"][row]).all() and torch.isnan(o["rstd_post"][row]), row
            else:  # only h is normalised: the residual is what it is, and the row's block still counts
                kept = torch.ones(H, dtype=torch.bool, device=dev)
                kept[row: row + times] = False
                assert torch.equal(o["ro"][row][kept], want["ro"][row][kept])
            if fmt in (R.MXFP4, R.NVFP4):  # every block of the row has a NaN scale
                sf = o["sf"].cpu().numpy()[R.sf_place(rows, -(-H // R.BLOCK[fmt]))][row]
                assert (sf == (255 if fmt == R.MXFP4 else 127)).all()
        assert torch.isnan(o["amax"]).all()
        # the norm before the next block alone
        if where == "residual":
            p = forward(d, rows, H, 5, 0.5, 1e-6, fmt=fmt, block=False, dev=dev)
            assert torch.equal(p["ro"].view(torch.int16), d["residual"].view(torch.int16))
            for row in (0, 4, 11):
                assert torch.isnan(p["h"][row]).all()


@pytest.mark.parametrize("H", [64, 4096, 16384])
def test_the_largest_rows_that_a_mean_holds(dev, H):
    """Squares that add up to just under binary32's largest: ordinary rows."""
    d = make(4, H, 4, None, 3, dev)
    d["residual"][1] = float((2.0 ** 128 * 0.9 / H) ** 0.5)
    d["residual"][3] = 0
    d["residual"][3, H // 2] = 2.0 ** 63.9
    o = forward(d, 4, H, 4, 1.0, 1e-6, block=False, dev=dev)
    v = d["residual"].double()
    h = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6) * d["pre"].double()
    assert ((o["h"].double() - h).abs() <= 2.0 ** -8 * 1.01 * h.abs()).all()
