"""The packed 4-bit operands on the GPU: quantize (of a matrix and of its transpose) bit for bit
against the definition in float64, dequantize bit for bit, and the product against float64 sums."""
import numpy as np
import pytest
import torch

import fp4_reference as R
from gpu_helpers import assert_bf16_equal, bf16_bits_of
from quantize_amax_scaling_gb300 import fp8q

pytestmark = pytest.mark.gpu
CANARY = 0xEE


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def from_bits(b, dev):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).to(dev).view(torch.bfloat16)


def inputs(r, c, seed, specials=False):
    """bf16 bits with a wide spread of block maxima, zero blocks, ties, and on request NaN and infinities."""
    rng = np.random.RandomState(seed)
    x = rng.standard_normal((r, c)) * np.exp2(rng.randint(-12, 6, (r, 1))) * np.exp2(rng.randint(-3, 4, (1, c)))
    x[rng.rand(r, c) < 0.1] *= 0
    ties = rng.rand(r, c) < 0.2
    x[ties] = (np.round(x * 4) / 4)[ties]
    x[:: 7, : 40] = 0
    if specials:
        for v in (np.nan, np.inf, -np.inf, 1e-40, -3e38, -0.0):
            x.reshape(-1)[rng.randint(0, x.size, 1 + x.size // 400)] = v
    return bf16_bits_of(torch.from_numpy(x).to(torch.bfloat16)).reshape(r, c)


def guarded_pair(r, c, fmt, dev):
    """A packed operand's arrays inside one canary-filled buffer each."""
    out = []
    for n in (r * fp8q.fp4_row_bytes(c), fp8q.fp4_scale_bytes(r, c, fmt)):
        buf = torch.full((n + 128,), CANARY, dtype=torch.uint8, device=dev)
        out += [buf, buf[64: 64 + n]]
    return out


def check_packed(qb, q, sb, s, bits, fmt, scale):
    r, c = bits.shape
    codes, sf, nan = R.quantize(bits, fmt, scale)
    want_q, want_s = R.pack(codes, sf)
    for buf, n in ((qb, q.numel()), (sb, s.numel())):
        raw = buf.cpu().numpy()
        assert (raw[:64] == CANARY).all() and (raw[64 + n:] == CANARY).all(), "write outside the operand"
    assert np.array_equal(s.cpu().numpy(), want_s), "block scales differ"
    got = q.cpu().numpy().reshape(r, -1)
    if nan.any():  # codes of a block that is NaN are free
        gc, _ = R.unpack(got, want_s, r, c, fmt)
        free = np.repeat(nan, R.BLOCK[fmt], axis=1)[:, :c]
        assert np.array_equal(gc[~free], codes[~free]), "codes differ"
        assert not (got.reshape(-1)[(want_q == 0).reshape(-1) & (np.arange(got.size) % got.shape[1] >= (c + 1) // 2)]).any()
    else:
        assert np.array_equal(got, want_q), "codes differ"


SHAPES = [(1, 1), (1, 16), (1, 4096), (3, 17), (5, 31), (33, 32), (64, 100), (127, 129), (128, 128), (129, 127), (130, 256),
          (1000, 48), (31, 2731), (257, 513), (640, 1040)]


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("r,c", SHAPES)
def test_quantize_both_ways(dev, r, c, fmt):
    bits = inputs(r, c, r * 7 + c)
    x = from_bits(bits, dev)
    scale = None if fmt == R.MXFP4 else 0.0123
    st = None if scale is None else torch.full((1,), scale, device=dev)
    qb, q, sb, s = guarded_pair(r, c, fmt, dev)
    tb, t, ub, u = guarded_pair(c, r, fmt, dev)
    amax = torch.zeros(1, device=dev)
    fp8q.fp8q_fp4_quantize_amax(x, q, s, fmt, st, amax, qt=t, sft=u)
    check_packed(qb, q, sb, s, bits, fmt, scale)
    check_packed(tb, t, ub, u, bits.T, fmt, scale)
    assert float(amax) == np.abs(R.bf16_to_f64(bits)).max()
    # one direction alone, without amax: the same bytes
    q2, s2 = torch.full_like(q, CANARY), torch.full_like(s, CANARY)
    t2, u2 = torch.full_like(t, CANARY), torch.full_like(u, CANARY)
    fp8q.fp8q_fp4_quantize_amax(x, q2, s2, fmt, st)
    fp8q.fp8q_fp4_quantize_amax(x, None, None, fmt, st, qt=t2, sft=u2)
    assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(t2, t) and torch.equal(u2, u)


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("off", [1, 8])
def test_quantize_from_any_address(dev, fmt, off):
    bits = inputs(70, 96, 5)
    room = torch.zeros(70 * 96 + 64, dtype=torch.bfloat16, device=dev)
    x = room[off: off + 70 * 96].view(70, 96)
    x.copy_(from_bits(bits, dev))
    qb, q, sb, s = guarded_pair(70, 96, fmt, dev)
    fp8q.fp8q_fp4_quantize_amax(x, q, s, fmt)
    check_packed(qb, q, sb, s, bits, fmt, None)


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
def test_quantize_specials(dev, fmt):
    bits = inputs(200, 333, 11, specials=True)
    x = from_bits(bits, dev)
    qb, q, sb, s = guarded_pair(200, 333, fmt, dev)
    tb, t, ub, u = guarded_pair(333, 200, fmt, dev)
    amax = torch.zeros(1, device=dev)
    fp8q.fp8q_fp4_quantize_amax(x, q, s, fmt, None, amax, qt=t, sft=u)
    check_packed(qb, q, sb, s, bits, fmt, None)
    check_packed(tb, t, ub, u, bits.T, fmt, None)
    assert torch.isnan(amax).all()


@pytest.mark.parametrize("scale", [1.0, 1 / 3, 2.0 ** -64, 2.0 ** -58, 1e-30, 1e-38, 1e-44, 2.0 ** 62, 3e37, 1e38, 0.0, -1.0,
                                   float("inf"), float("nan")])
def test_nvfp4_every_bf16_at_many_scales(dev, scale):
    bits = np.arange(65536, dtype=np.uint16)
    with np.errstate(invalid="ignore"):
        ordinary = ~np.isnan(R.bf16_to_f64(bits))
    bits = np.resize(bits[ordinary], (510, 128 * 16 // 16))  # neighbours share a block
    x = from_bits(bits, dev)
    qb, q, sb, s = guarded_pair(*bits.shape, R.NVFP4, dev)
    fp8q.fp8q_fp4_quantize_amax(x, q, s, R.NVFP4, torch.full((1,), scale, device=dev))
    check_packed(qb, q, sb, s, bits, R.NVFP4, scale)


def test_mxfp4_every_bf16_with_every_maximum(dev):
    """Each row: a block maximum of another exponent, and values down to those that vanish against it."""
    tops = (np.arange(0, 256, dtype=np.uint16) << 7) | 0x55
    tops = tops[tops < 0x7F80]
    rows = [np.concatenate([np.clip(np.arange(t - 31, t + 1), 0, 0x7F7F), np.clip(np.arange(t - 992, t, 32), 0, 0x7F7F)])
            for t in tops.astype(np.int64)]
    bits = np.stack(rows).astype(np.uint16)
    bits[:, 1::2] |= 0x8000
    qb, q, sb, s = guarded_pair(*bits.shape, R.MXFP4, dev)
    fp8q.fp8q_fp4_quantize_amax(from_bits(bits, dev), q, s, R.MXFP4)
    check_packed(qb, q, sb, s, bits, R.MXFP4, None)


def random_operand(r, c, fmt, seed, dev, sf_lo=None, sf_hi=None):
    """Codes and scales drawn directly; scale bytes of no row hold 0xFF: a NaN in either format."""
    rng = np.random.RandomState(seed)
    codes = rng.randint(0, 16, (r, c)).astype(np.uint8)
    lo, hi = (sf_lo, sf_hi) if sf_lo is not None else ((120, 134) if fmt == R.MXFP4 else (0x20, 0x50))
    sf = rng.randint(lo, hi, (r, -(-c // R.BLOCK[fmt]))).astype(np.uint8)
    q, s = R.pack(codes, sf)
    s[s == 0xEE] = 0xFF
    place = R.sf_place(r, -(-sf.shape[1] // 4) * 4)
    t = np.full_like(s, 0xFF)
    t[place] = 0
    t[R.sf_place(r, sf.shape[1])] = sf
    return torch.from_numpy(q).to(dev), torch.from_numpy(t).to(dev), codes, sf


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("r,c", SHAPES)
def test_dequantize(dev, r, c, fmt):
    q, s, codes, sf = random_operand(r, c, fmt, r + c, dev, 0, 256 if fmt == R.MXFP4 else 0x80)
    for scale in (None,) if fmt == R.MXFP4 else (None, 0.37, 1e-30):
        y = torch.full((r * c + 64,), 7.0, dtype=torch.bfloat16, device=dev)
        fp8q.fp8q_fp4_dequantize(q, s, y[32: 32 + r * c].view(r, c), fmt, None if scale is None else torch.full((1,), scale, device=dev))
        with np.errstate(all="ignore"):
            want = R.values(codes, sf, fmt, None).astype(np.float32)  # exact
            if scale is not None:
                want = want * np.float32(scale)
        assert (y[:32] == 7).all() and (y[32 + r * c:] == 7).all()
        assert_bf16_equal(bf16_bits_of(y[32: 32 + r * c]), bf16_bits_of(torch.from_numpy(want).to(torch.bfloat16)))


MATMULS = [(1, 1, 1), (1, 8, 16), (1, 4096, 4096), (2, 130, 31), (3, 1000, 257), (7, 16, 16384), (8, 129, 64), (16, 256, 96),
           (17, 300, 130), (24, 512, 2048), (33, 77, 640), (64, 128, 65), (65, 200, 1033), (100, 333, 333), (128, 128, 128), (129, 257, 192),
           (255, 256, 256), (256, 512, 320), (300, 1000, 1033), (513, 520, 1024), (1024, 768, 4096), (1555, 640, 257), (2048, 1, 512),
           (4096, 40, 72), (640, 2056, 1536), (2000, 2304, 96),
           (2100, 2050, 257), (4100, 1104, 1056), (200, 17000, 96), (2304, 2400, 640), (1030, 4099, 33)]


def product_bound(a, b, want, k, alpha, out_eps):
    """|error| allowed: k binary32 additions, each off by at most one unit in the last place (2^-23 of a
    partial sum, which the sum of |products| bounds), two roundings by the scales (2^-24 each), and half a step of the output type."""
    mag = (a.abs() @ b.abs().t()) * alpha
    return (k * 2.0 ** -23 + 2.0 ** -23) * mag + out_eps / 2 * want.abs() + 2.0 ** -133


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("m,n,k", MATMULS)
def test_matmul(dev, m, n, k, fmt):
    qa, sa, ca, fa = random_operand(m, k, fmt, m + n + k, dev)
    qb, sb, cb, fb = random_operand(n, k, fmt, m + n + k + 1, dev)
    a = torch.from_numpy(R.values(ca, fa, fmt)).to(dev)
    b = torch.from_numpy(R.values(cb, fb, fmt)).to(dev)
    scales = (None, None) if fmt == R.MXFP4 else (torch.full((1,), 0.013, device=dev), torch.full((1,), 1.7, device=dev))
    alpha = 1.0 if fmt == R.MXFP4 else float(scales[0].double() * scales[1].double())
    want = (a @ b.t()) * alpha
    for dtype, eps in ((torch.bfloat16, 2.0 ** -7), (torch.float32, 2.0 ** -23)):
        room = torch.full((m * n + 64,), 7.0, dtype=dtype, device=dev)
        d = room[32: 32 + m * n].view(m, n)
        fp8q.fp8q_fp4_matmul(qa, sa, qb, sb, d, k, fmt, *scales)
        assert (room[:32] == 7).all() and (room[32 + m * n:] == 7).all(), "write outside the product"
        off = (d.double() - want).abs()
        bad = off > product_bound(a, b, want, k, alpha, eps)
        assert not bad.any(), f"{int(bad.sum())} of {m * n} off, first at {bad.nonzero()[0].tolist()}: {float(off[bad][0])}"
        again = torch.empty_like(d)
        fp8q.fp8q_fp4_matmul(qa, sa, qb, sb, again, k, fmt, *scales)
        assert torch.equal(again, d), "the same call gave other bits"


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("m,n,k", [(1, 640, 4096), (5, 384, 1000), (40, 256, 8192), (200, 300, 2048), (700, 1100, 1056), (512, 512, 512),
                                   (2300, 2112, 1100), (2200, 2051, 2048), (16384, 520, 256), (2560, 8192, 128)])
def test_matmul_exact_sums(dev, m, n, k, fmt):
    """Scales of 1, 2 and 4 and few enough terms: every partial sum is a multiple of 1/4 below 2^22, exact in
    binary32 in any order, so the product is exact: a wrong code, scale or place shows in the last bit."""
    lo, hi = (127, 130) if fmt == R.MXFP4 else (0x38, 0x39)  # e4m3 0x38 is 1
    qa, sa, ca, fa = random_operand(m, k, fmt, k + 1, dev, lo, hi)
    qb, sb, cb, fb = random_operand(n, k, fmt, k + 2, dev, lo, hi)
    if fmt == R.NVFP4:  # 1, 2 or 4
        rng = np.random.RandomState(k)
        for s, f, rows in ((sa, fa, m), (sb, fb, n)):
            f[:] = rng.choice([0x38, 0x40, 0x48], f.shape)
            s[torch.from_numpy(R.sf_place(*f.shape)).to(dev)] = torch.from_numpy(f).to(dev)
    a = torch.from_numpy(R.values(ca, fa, fmt)).to(dev)
    b = torch.from_numpy(R.values(cb, fb, fmt)).to(dev)
    assert float((a.abs() @ b.abs().t()).max()) < 2 ** 22
    d = torch.empty((m, n), device=dev)
    fp8q.fp8q_fp4_matmul(qa, sa, qb, sb, d, k, fmt)
    assert torch.equal(d.double(), a @ b.t())


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("m,n,k", [(1100, 2305, 2100), (2600, 2571, 100), (2600, 2701, 100), (2600, 2574, 100)])
def test_matmul_odd_rows(dev, m, n, k, fmt):
    """Rows of D that start anywhere, on single CTAs and on pairs."""
    test_matmul(dev, m, n, k, fmt)


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("m,n,k", [(2, 9800, 8192), (16, 4097, 2048), (9, 300, 4100), (24, 9800, 8200), (24, 6000, 4097), (30, 335, 16384),
                                   (64, 8200, 4200), (64, 4097, 3000), (60, 1001, 8200), (256, 4096, 8192), (128, 4097, 4096),
                                   (300, 1000, 4096), (128, 1024, 8192), (100, 333, 4100)])
def test_matmul_sums_shared_by_clusters(dev, m, n, k, fmt):
    """Clusters of 2, 4 and 8 for each width of tile, rows of D that hold whole vectors and odd ones, exact sums."""
    test_matmul_exact_sums(dev, m, n, k, fmt)


@pytest.mark.parametrize("m,n,k", [(3, 64, 96), (300, 520, 320)])
def test_matmul_nan_block_reaches_its_row_only(dev, m, n, k):
    qa, sa, ca, fa = random_operand(m, k, R.MXFP4, 1, dev)
    qb, sb, cb, fb = random_operand(n, k, R.MXFP4, 2, dev)
    sa[int(R.sf_place(m, -(-k // 32))[m - 1, 1])] = 255
    d = torch.empty((m, n), device=dev)
    fp8q.fp8q_fp4_matmul(qa, sa, qb, sb, d, k, R.MXFP4)
    assert torch.isnan(d[m - 1]).all() and not torch.isnan(d[: m - 1]).any()


def test_empty_calls_launch_nothing(dev):
    q, s = fp8q.fp4_empty(0, 64, R.NVFP4, dev)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=dev)
    fp8q.fp8q_fp4_quantize_amax(x, q, s, R.NVFP4)
    fp8q.fp8q_fp4_dequantize(q, s, x, R.NVFP4)
    b = fp8q.fp4_empty(5, 64, R.NVFP4, dev)
    fp8q.fp8q_fp4_matmul(q, s, *b, torch.empty((0, 5), dtype=torch.bfloat16, device=dev), 64, R.NVFP4)
    with pytest.raises(ValueError):
        fp8q.fp8q_fp4_quantize_amax(torch.zeros((4, 33), dtype=torch.bfloat16, device=dev), *fp8q.fp4_empty(4, 32, R.NVFP4, dev), R.NVFP4)
    with pytest.raises(fp8q.Fp8qError):
        fp8q.fp8q_fp4_quantize_amax(torch.zeros((4, 32), dtype=torch.bfloat16, device=dev), *fp8q.fp4_empty(4, 32, R.MXFP4, dev), R.MXFP4,
                                    torch.ones(1, device=dev))


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
def test_on_another_stream_and_in_a_graph(dev, fmt):
    """Quantize and multiply on a side stream and replayed from a CUDA graph with new inputs: the eager results."""
    m, n, k = 70, 200, 300
    x = [from_bits(inputs(m, k, 90 + i), dev) for i in range(3)]
    w = from_bits(inputs(n, k, 99), dev)
    wp = fp8q.fp4_empty(n, k, fmt, dev)
    fp8q.fp8q_fp4_quantize_amax(w, *wp, fmt)

    def step(inp, p, d, **kw):
        fp8q.fp8q_fp4_quantize_amax(inp, *p, fmt, **kw)
        fp8q.fp8q_fp4_matmul(*p, *wp, d, k, fmt, **kw)

    want = []
    for t in x:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
        step(t, fp8q.fp4_empty(m, k, fmt, dev), d)
        want.append(d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    d, p = torch.empty_like(want[0]), fp8q.fp4_empty(m, k, fmt, dev)
    step(x[1], p, d, stream=side)
    side.synchronize()
    assert torch.equal(d, want[1])
    inp = x[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(inp, p, d)
    for t, y in zip(x, want):
        inp.copy_(t)
        d.zero_()
        g.replay()
        assert torch.equal(d, y)


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("m,n,k", [(64, 16384, 4096), (1100, 4352, 2816)])
def test_matmul_from_cold_memory(dev, m, n, k, fmt):
    """Operands that come from memory in any order, many calls one behind another: the same exact sums each time."""
    g = torch.Generator(device=dev)
    g.manual_seed(k)
    one = 127 if fmt == R.MXFP4 else 0x38
    grid = torch.tensor(R.VALUE, dtype=torch.float32, device=dev)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=dev)
    sets = []
    for _ in range(3):
        ops, vals = [], []
        for r in (m, n):
            q, s = fp8q.fp4_empty(r, k, fmt, dev)
            q.copy_(torch.randint(0, 256, q.shape, generator=g, device=dev, dtype=torch.uint8))
            s.fill_(one)
            ops.append((q, s))
            vals.append(grid[torch.stack((q & 15, q >> 4), -1).view(r, -1)[:, :k].int()])
        sets.append((ops, vals[0].double() @ vals[1].double().t()))
    d = [torch.empty((m, n), device=dev) for _ in sets]
    for i in range(10):
        flush.zero_()
        for (ops, _), out in zip(sets, d):
            fp8q.fp8q_fp4_matmul(*ops[0], *ops[1], out, k, fmt)
        for (_, want), out in zip(sets, d):
            assert torch.equal(out.double(), want)
