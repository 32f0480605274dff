"""The FP8 products grouped by expert, and the experts' weight gradients, on the GPU: each group against the product of its
rows alone, rows of no group left as they were, and nothing of one group's codes in another's sums."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_matmul import check, gen, guarded, stored, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def experts(e, rows, cols, fmt, g, trans=False):
    """[e, rows, cols] codes, and as the call takes them (each matrix transposed in memory on request)."""
    w = R.random_codes((e, rows, cols), fmt, g)
    t = w.transpose(1, 2).contiguous() if trans else w
    ld = (t.shape[2] + 15) // 16 * 16
    room = torch.full((e, t.shape[1], ld), 0x7F, dtype=torch.uint8, device=w.device)
    room[:, :, : t.shape[2]] = t
    return w, room[:, :, : t.shape[2]]


# few rows a group (CTAs of 16 to 128 rows) and many (pairs of CTAs of 256): empty groups, one row, ends inside tiles,
# rows before the first and behind the last
GROUPS = [[0, 1], [0, 0, 0], [3, 3, 9, 9, 30, 31, 40], [0, 16, 32, 33, 33, 90], [5, 133, 133, 400, 401, 700], [0, 129, 129, 130, 1000, 1300],
          [0, 256, 512, 513, 769, 1025], [0] * 40 + [7] + [500] * 60 + [900] * 30, list(range(0, 512, 4)), [100, 2100, 2100, 2399]]


def extent(off):
    return off[-1] + (11 if off[0] else 0)


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("n,k", [(130, 100), (640, 272), (257, 1040)])
@pytest.mark.parametrize("off", GROUPS, ids=lambda o: f"{len(o) - 1}of{o[-1]}")
def test_rows(dev, off, n, k, tb):
    e, rows = len(off) - 1, extent(off)
    g = gen(dev, rows + n + k)
    a = R.random_codes((rows, k), 1, g)
    w, wt = experts(e, n, k, 0, g, tb)
    bias = torch.randn((e, n), generator=g, device=dev)
    at = torch.tensor(off, dtype=torch.int32, device=dev)
    s = torch.full((1,), 1.0 / k ** 0.5, device=dev)
    buf, d = guarded((rows, n), torch.float32, dev)
    d.fill_(77.0)
    fp8q.fp8q_grouped_matmul(stored(a, 0), wt, at, d, 1, 0, s, None, b_trans=tb, bias=bias)
    whole(buf)
    inside = torch.zeros(rows, dtype=torch.bool, device=dev)
    for i in range(e):
        lo, hi = off[i], off[i + 1]
        inside[lo:hi] = True
        if lo < hi:
            va, vb = R.values(a[lo:hi], 1), R.values(w[i], 0)
            want = va @ vb.t() * float(s) + bias[i].double()
            check(d[lo:hi], want, R.sum_bound(va, vb) * float(s) + 2.0 ** -23 * want.abs())
    assert (d[~inside] == 77.0).all(), "a row of no group was written"
    # every other part of the epilogue, from the same sums
    res = torch.randn((rows, n), generator=g, device=dev).to(torch.bfloat16)
    y, q, amax = torch.full((rows, n), 5.0, dtype=torch.bfloat16, device=dev), torch.full((rows, n), 9, dtype=torch.uint8, device=dev), torch.zeros(1, device=dev)
    h, sf = (t.fill_(3) for t in fp8q.checkpoint_empty(rows, n))
    fp8q.fp8q_grouped_matmul(stored(a, 0), wt, at, y, 1, 0, s, None, b_trans=tb, bias=bias, act=1, residual=res, q=q, q_scale=s, amax=amax, h=h, h_sf=sf)
    z = torch.zeros((rows, n), dtype=torch.bfloat16, device=dev)
    fp8q.fp8q_grouped_matmul(stored(a, 0), wt, at, z, 1, 0, s, None, b_trans=tb, bias=bias)
    assert torch.equal(z[inside], d[inside].to(torch.bfloat16))
    q2, h2, sf2 = torch.empty_like(q), torch.empty_like(h), torch.empty_like(sf)
    fp8q.fp8q_quantize_amax(y, q2, 0, s, torch.zeros(1, device=dev))
    fp8q.fp8q_checkpoint_quantize(z, h2, sf2)
    for got, want, old in ((q, q2, 9), (h, h2, 3), (sf, sf2, 3)):
        assert torch.equal(got[inside], want[inside]) and (got[~inside] == old).all()
    assert (y[~inside] == 5.0).all()
    assert float(amax) == (float(y[inside].float().abs().max()) if inside.any() else 0.0)
    want = R.gelu(d[inside].double()) + res[inside].double()
    assert ((y[inside].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * (want - res[inside].double()).abs() + 2.0 ** -22 * res[inside].double().abs() + 2.0 ** -60).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(130, 100), (256, 640), (517, 1040)])
@pytest.mark.parametrize("off", GROUPS, ids=lambda o: f"{len(o) - 1}of{o[-1]}")
def test_weight_gradients(dev, off, m, n, dtype):
    e, rows = len(off) - 1, extent(off)
    g = gen(dev, rows + m + n)
    a, b = R.random_codes((rows, m), 1, g), R.random_codes((rows, n), 0, g)
    at = torch.tensor(off, dtype=torch.int32, device=dev)
    s = torch.full((1,), 0.03, device=dev)
    buf, d = guarded((e, m, n), dtype, dev)
    fp8q.fp8q_grouped_weight_gradient(stored(a, 0), stored(b, 0, 1), at, d, 1, 0, s, None)
    whole(buf)
    for i in range(e):
        va, vb = R.values(a[off[i]: off[i + 1]], 1).t(), R.values(b[off[i]: off[i + 1]], 0).t()
        check(d[i], va @ vb.t() * float(s), R.sum_bound(va, vb) * float(s))
    # added to what is there, in place
    old = torch.randn((e, m, n), generator=g, device=dev).to(dtype)
    buf, d2 = guarded((e, m, n), dtype, dev)
    d2.copy_(old)
    fp8q.fp8q_grouped_weight_gradient(stored(a, 0), stored(b, 0), at, d2, 1, 0, s, None, residual=d2)
    whole(buf)
    for i in range(e):
        va, vb = R.values(a[off[i]: off[i + 1]], 1).t(), R.values(b[off[i]: off[i + 1]], 0).t()
        want = va @ vb.t() * float(s) + old[i].double()
        check(d2[i], want, R.sum_bound(va, vb) * float(s) + 2.0 ** -23 * want.abs())


@pytest.mark.parametrize("cut", [1, 31, 32, 33, 127, 128, 129, 200])
def test_nan_of_another_group_stays_there(dev, cut):
    """NaN codes in the rows around a group, in either operand, do not reach its gradient or its rows."""
    rows, m, n = 400, 200, 300
    g = gen(dev, cut)
    a, b = R.random_codes((rows, m), 0, g), R.random_codes((rows, n), 0, g)
    w, wt = experts(3, n, 208, 0, g)
    x = R.random_codes((rows, 208), 0, g)
    lo = 60
    for t in (a, b, x):
        t[:lo] = 0x7F
        t[lo + cut:] = 0xFF
    w[0], w[2] = 0x7F, 0x7F
    at = torch.tensor([0, lo, lo + cut, rows], dtype=torch.int32, device=dev)
    d = torch.empty((3, m, n), device=dev)
    fp8q.fp8q_grouped_weight_gradient(stored(a, 0), stored(b, 0), at, d)
    va, vb = R.values(a[lo: lo + cut], 0).t(), R.values(b[lo: lo + cut], 0).t()
    a8 = torch.empty_like(d)
    fp8q.fp8q_grouped_weight_gradient(stored(a, 0), stored(b, 0), at, a8, 0, 0)
    check(a8[1], va @ vb.t(), R.sum_bound(va, vb))
    assert torch.isnan(a8[0]).all() and torch.isnan(a8[2]).all()
    y = torch.empty((rows, n), device=dev)
    fp8q.fp8q_grouped_matmul(x, w, at, y)
    va, vb = R.values(x[lo: lo + cut], 0), R.values(w[1], 0)
    check(y[lo: lo + cut], va @ vb.t(), R.sum_bound(va, vb))
    assert torch.isnan(y[:lo]).all() and torch.isnan(y[lo + cut:]).all()


def test_more_rows_than_a_step_and_more_tiles_than_pairs(dev):
    """Groups of unlike lengths over more tiles than pairs of CTAs, so that stages and accumulators come round many times."""
    g = gen(dev, 9)
    off = [0, 1500, 1500, 1777, 3333, 3334]
    rows, m, n = off[-1], 1280, 1536
    a, b = R.random_codes((rows, m), 1, g), R.random_codes((rows, n), 0, g)
    at = torch.tensor(off, dtype=torch.int32, device=dev)
    d = torch.empty((5, m, n), device=dev)
    fp8q.fp8q_grouped_weight_gradient(a, b, at, d)
    for i in range(5):
        va, vb = R.values(a[off[i]: off[i + 1]], 1).t(), R.values(b[off[i]: off[i + 1]], 0).t()
        check(d[i], va @ vb.t(), R.sum_bound(va, vb))
    w, _ = experts(5, 4096, m, 0, g)
    y = torch.empty((rows, 4096), dtype=torch.bfloat16, device=dev)
    fp8q.fp8q_grouped_matmul(a, w, at, y, 1, 0)
    for i in range(5):
        if off[i] < off[i + 1]:
            va, vb = R.values(a[off[i]: off[i + 1]], 1), R.values(w[i], 0)
            check(y[off[i]: off[i + 1]], va @ vb.t(), R.sum_bound(va, vb))


@pytest.mark.parametrize("off", [[0, 50, 20, 70, 300], [-5, 40, 90, 1000, 2000000000], [300, 200, 100, 50, 0], [-2 ** 31, 2 ** 31 - 1, -1, 299, 2 ** 31 - 1]])
@pytest.mark.parametrize("rows", [300, 1300])
def test_offsets_that_are_wrong_stay_in_bounds(dev, off, rows):
    """Whatever the offsets say, nothing outside the outputs is written; groups that are well formed among them are right."""
    g = gen(dev, 2)
    a, (w, _) = R.random_codes((rows, 64), 0, g), experts(4, 200, 64, 0, g)
    at = torch.tensor(off, dtype=torch.int32, device=dev)
    buf, y = guarded((rows, 200), torch.float32, dev)
    y.fill_(3.0)
    fp8q.fp8q_grouped_matmul(a, w, at, y)
    whole(buf)
    inside = torch.zeros(rows, dtype=torch.int32, device=dev)
    for i in range(4):
        lo, hi = max(0, min(off[i], rows)), max(0, min(off[i + 1], rows))
        if lo < hi:
            inside[lo:hi] += 1
    assert (y[inside == 0] == 3.0).all()
    buf, d = guarded((4, 64, 64), torch.float32, dev)
    fp8q.fp8q_grouped_weight_gradient(a, a, at, d, 0, 0)
    whole(buf)
    for i in range(4):
        lo, hi = max(0, min(off[i], rows)), max(0, min(off[i + 1], rows))
        v = R.values(a[lo: max(lo, hi)], 0).t()
        check(d[i], v @ v.t(), R.sum_bound(v, v))


def test_nothing(dev):
    at = torch.zeros(4, dtype=torch.int32, device=dev)
    empty = torch.empty((0, 32), dtype=torch.uint8, device=dev)
    d = torch.full((3, 32, 32), 5.0, device=dev)
    old = d.clone()
    fp8q.fp8q_grouped_weight_gradient(empty, empty, at, d)
    assert not d.any()
    fp8q.fp8q_grouped_weight_gradient(empty, empty, at, d, residual=old)
    assert torch.equal(d, old)
    w = torch.zeros((3, 16, 32), dtype=torch.uint8, device=dev)
    fp8q.fp8q_grouped_matmul(empty, w, at, torch.empty((0, 16), device=dev))
    # no groups: no rows of any
    x, y = torch.zeros((5, 32), dtype=torch.uint8, device=dev), torch.full((5, 16), 2.0, device=dev)
    fp8q.fp8q_grouped_matmul(x, w[:0], at[:1], y)
    assert (y == 2.0).all()
    # groups of an empty k: bias alone
    bias = torch.randn((3, 16), device=dev)
    at = torch.tensor([0, 2, 2, 4], dtype=torch.int32, device=dev)
    fp8q.fp8q_grouped_matmul(x[:, :0].contiguous(), w[:, :, :0].contiguous(), at, y, bias=bias)
    assert torch.equal(y, torch.stack([bias[0], bias[0], bias[2], bias[2], torch.full((16,), 2.0, device=dev)]))


@pytest.mark.parametrize("rows,e", [(40, 8), (3000, 6)])
def test_replayed_with_other_offsets(dev, rows, e):
    """A captured call reads the offsets of each replay."""
    g = gen(dev, 5)
    a, (w, _) = R.random_codes((rows, 128), 1, g), experts(e, 256, 128, 0, g)
    at = torch.zeros(e + 1, dtype=torch.int32, device=dev)
    y, d = torch.zeros((rows, 256), device=dev), torch.empty((e, 128, 256), device=dev)

    def call(y, d):
        fp8q.fp8q_grouped_matmul(a, w, at, y, 1, 0)
        fp8q.fp8q_grouped_weight_gradient(a, y.to(torch.float8_e4m3fn).view(torch.uint8), at, d, 1, 0)

    call(y, d)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call(y, d)
    for seed in range(3):
        cut = torch.randint(0, rows + 1, (e - 1,), generator=gen(dev, seed), device=dev).sort().values.to(torch.int32)
        at[1:e], at[e] = cut, rows
        gr.replay()
        y2, d2 = torch.zeros_like(y), torch.empty_like(d)
        call(y2, d2)
        assert torch.equal(y, y2) and torch.equal(d, d2)


def test_refusals(dev):
    a, w = torch.zeros((8, 32), dtype=torch.uint8, device=dev), torch.zeros((3, 16, 32), dtype=torch.uint8, device=dev)
    y, at = torch.empty((8, 16), device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
    good = dict(a=a, b=w, offsets=at, d=y)
    fp8q.fp8q_grouped_matmul(**good)
    for bad in (dict(offsets=at[:3]), dict(offsets=at.long()), dict(offsets=None), dict(b=w[0]), dict(b=w[:, ::2]), dict(bias=torch.zeros(16, device=dev)),
                dict(d=y[:7]), dict(offsets=at.cpu())):
        with pytest.raises(ValueError):
            fp8q.fp8q_grouped_matmul(**{**good, **bad})
    many = torch.zeros((513, 16, 32), dtype=torch.uint8, device=dev)
    with pytest.raises(fp8q.Fp8qError) as err:
        fp8q.fp8q_grouped_matmul(a, many, torch.zeros(514, dtype=torch.int32, device=dev), y)
    assert err.value.status == 2
    d = torch.empty((3, 32, 16), device=dev)
    b = torch.zeros((8, 16), dtype=torch.uint8, device=dev)
    fp8q.fp8q_grouped_weight_gradient(a, b, at, d)
    for bad in (dict(d=d[:2]), dict(d=d[0]), dict(b=b[:7]), dict(residual=d.bfloat16()), dict(offsets=None)):
        with pytest.raises(ValueError):
            fp8q.fp8q_grouped_weight_gradient(**{**dict(a=a, b=b, offsets=at, d=d), **bad})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(272, 1040), (1040, 2064)])
def test_gradients_on_top_over_many_tiles(dev, m, n, dtype):
    """Added to what is there: bit for bit the sum of it and of the call without it, over more tiles than pairs of CTAs, empty
    groups among them; and rows by expert with a residual the same."""
    off = [0, 0, 40, 41, 300, 300, 428, 700, 701, 1000, 1300, 1300, 1301, 1500, 1501, 1502, 2000, 2000, 2100]
    e, rows = len(off) - 1, off[-1]
    g = gen(dev, m + n)
    a, b = R.random_codes((rows, m), 1, g), R.random_codes((rows, n), 0, g)
    at = torch.tensor(off, dtype=torch.int32, device=dev)
    s = torch.full((1,), 0.03, device=dev)
    plain = torch.empty((e, m, n), device=dev)
    fp8q.fp8q_grouped_weight_gradient(a, b, at, plain, 1, 0, s, None)
    old = torch.randn((e, m, n), generator=g, device=dev).to(dtype)
    buf, d = guarded((e, m, n), dtype, dev)
    d.copy_(old)
    fp8q.fp8q_grouped_weight_gradient(a, b, at, d, 1, 0, s, None, residual=d)
    whole(buf)
    assert torch.equal(d, (plain + old.float()).to(dtype))
    few = torch.tensor([7, 7, 900, 901, 2093], dtype=torch.int32, device=dev)
    w, wt = experts(4, n, m, 0, g)
    y, old = torch.zeros((rows, n), device=dev), torch.randn((rows, n), generator=g, device=dev).to(dtype)
    fp8q.fp8q_grouped_matmul(a, wt, few, y, 1, 0, s, None)
    buf, d = guarded((rows, n), dtype, dev)
    d.copy_(old)
    fp8q.fp8q_grouped_matmul(a, wt, few, d, 1, 0, s, None, residual=d)
    whole(buf)
    assert torch.equal(d, (y + old.float()).to(dtype))
