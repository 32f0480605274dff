"""The FP8 product and its epilogue on the GPU: sums against float64 in every orientation, and each part of the epilogue
either against float64 or, where another call defines it, bit for bit against that call."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q

pytestmark = pytest.mark.gpu
CANARY = 0xEE


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def stored(codes, trans, pad=0):
    """The matrix as the call takes it: transposed in memory on request, rows a multiple of 16 bytes apart (``pad`` 16s more)."""
    t = codes.t() if trans else codes
    ld = (t.shape[1] + 15) // 16 * 16 + 16 * pad
    room = torch.full((t.shape[0], ld), 0x7F, dtype=torch.uint8, device=codes.device)  # NaN between the rows
    room[:, : t.shape[1]] = t
    return room[:, : t.shape[1]]


def guarded(shape, dtype, dev):
    """A canary-filled buffer and the output within it."""
    n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
    buf = torch.full((n + 256,), CANARY, dtype=torch.uint8, device=dev)
    return buf, buf[128: 128 + n].view(dtype).view(shape)


def whole(buf):
    assert (buf[:128] == CANARY).all() and (buf[-128:] == CANARY).all(), "write outside the output"


def operands(dev, m, n, k, seed, fa=0, fb=0):
    g = gen(dev, seed)
    return R.random_codes((m, k), fa, g), R.random_codes((n, k), fb, g)


def check(got, want, bound):
    """Within the bound on the sums and half a step of the output's type (and half its least subnormal)."""
    err = (got.double() - want).abs()
    ok = err <= bound + R.HALF[got.dtype] * (want.abs() + bound) + 2.0 ** -134
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()} off, worst {float((err - bound).max())}"


# one token and few, tiles that end inside, both kernels, sums shared by clusters, more tiles than pairs of CTAs
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 640, 4096), (3, 17, 33), (16, 200, 1040), (17, 130, 160), (33, 256, 8192), (65, 200, 1033), (127, 129, 500),
          (128, 128, 31), (129, 257, 96), (200, 72, 4100), (300, 520, 320), (2560, 2304, 1100), (2561, 2308, 129), (3000, 2751, 64)]


@pytest.mark.parametrize("ta,tb", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_sums(dev, m, n, k, ta, tb):
    fa, fb = (m + ta) % 2, (n + tb) % 2
    a, b = operands(dev, m, n, k, m + 3 * n + 7 * k, fa, fb)
    va, vb = R.values(a, fa), R.values(b, fb)
    sa, sb = torch.full((1,), 0.37, device=dev), torch.full((1,), 1.9, device=dev)
    alpha = float(sa * sb)
    buf, d = guarded((m, n), torch.float32, dev)
    fp8q.fp8q_matmul(stored(a, ta, m % 3), stored(b, tb, n % 2), d, fa, fb, sa, sb, a_trans=ta, b_trans=tb)
    whole(buf)
    check(d, va @ vb.t() * alpha, R.sum_bound(va, vb) * alpha)
    buf2, d2 = guarded((m, n), torch.bfloat16, dev)
    fp8q.fp8q_matmul(stored(a, ta), stored(b, tb), d2, fa, fb, sa, sb, a_trans=ta, b_trans=tb)
    whole(buf2)
    assert torch.equal(d2, d.to(torch.bfloat16)), "bf16 is not the rounding of the float32 result"


@pytest.mark.parametrize("fa", [0, 1])
@pytest.mark.parametrize("fb", [0, 1])
@pytest.mark.parametrize("m,n,k", [(5, 130, 256), (2560, 2304, 256)])
def test_every_code(dev, m, n, k, fa, fb):
    """All finite codes of both formats, subnormals and the largest among them, against each other."""
    g = gen(dev, 3)
    a = torch.randint(0, 256, (m, k), generator=g, device=dev, dtype=torch.uint8)
    b = torch.randint(0, 256, (n, k), generator=g, device=dev, dtype=torch.uint8)
    a[~torch.isfinite(R.values(a, fa))] = 0x3A
    b[~torch.isfinite(R.values(b, fb))] = 0x81
    va, vb = R.values(a, fa), R.values(b, fb)
    d = torch.empty((m, n), device=dev)
    fp8q.fp8q_matmul(a, b, d, fa, fb)
    check(d, va @ vb.t(), R.sum_bound(va, vb))


EPILOGUE = [(1, 640, 512), (24, 200, 4096), (40, 133, 96), (130, 260, 160), (2600, 2304, 160), (2600, 2310, 48), (2600, 2307, 32)]


@pytest.mark.parametrize("bias_type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", EPILOGUE)
def test_bias_gelu_residual(dev, m, n, k, bias_type):
    a, b = operands(dev, m, n, k, 5)
    g = gen(dev, 6)
    bias = torch.randn(n, generator=g, device=dev).to(bias_type)
    va, vb = R.values(a, 0), R.values(b, 0)
    s = torch.full((1,), 0.5 / k ** 0.5, device=dev)
    z = va @ vb.t() * float(s) + bias.double()
    off = R.sum_bound(va, vb) * float(s) + 2.0 ** -23 * z.abs()
    A, B = stored(a, 0), stored(b, 0)
    for out in (torch.float32, torch.bfloat16):
        res = torch.randn((m, n), generator=g, device=dev).to(out)
        for act, residual in ((0, None), (1, None), (0, res), (1, res)):
            buf, d = guarded((m, n), out, dev)
            fp8q.fp8q_matmul(A, B, d, a_scale=s, bias=bias, act=act, residual=residual)
            whole(buf)
            want = R.gelu(z) if act else z
            bound = 1.13 * off + 2.0 ** -18 * want.abs() + 2.0 ** -100 if act else off
            if residual is not None:
                want = want + residual.double()
                bound = bound + 2.0 ** -23 * want.abs()
            check(d, want, bound)
        # in place
        buf, d = guarded((m, n), out, dev)
        d.copy_(res)
        fp8q.fp8q_matmul(A, B, d, a_scale=s, bias=bias, act=1, residual=d)
        whole(buf)
        ref = torch.empty_like(d)
        fp8q.fp8q_matmul(A, B, ref, a_scale=s, bias=bias, act=1, residual=res)
        assert torch.equal(d, ref)


@pytest.mark.parametrize("q_fmt", [0, 1])
@pytest.mark.parametrize("scale", [0.011, 2.0 ** -70, 1e30])
@pytest.mark.parametrize("m,n,k", EPILOGUE)
def test_codes_amax_and_checkpoint(dev, m, n, k, q_fmt, scale):
    """Bit for bit what the calls that define them make of the bf16 outputs."""
    a, b = operands(dev, m, n, k, 8)
    g = gen(dev, 9)
    A, B = stored(a, 0), stored(b, 0)
    bias = torch.randn(n, generator=g, device=dev)
    res = torch.randn((m, n), generator=g, device=dev).to(torch.bfloat16)
    s, qs = torch.full((1,), 1.0 / k ** 0.5, device=dev), torch.full((1,), scale, device=dev)
    z, y = (torch.empty((m, n), dtype=torch.bfloat16, device=dev) for _ in range(2))
    fp8q.fp8q_matmul(A, B, z, a_scale=s, bias=bias)
    fp8q.fp8q_matmul(A, B, y, a_scale=s, bias=bias, act=1, residual=res)
    want_q, want_amax = torch.empty((m, n), dtype=torch.uint8, device=dev), torch.full((1,), 0.25, device=dev)
    fp8q.fp8q_quantize_amax(y, want_q, q_fmt, qs, want_amax)
    want_h, want_sf = fp8q.checkpoint_empty(m, n)
    fp8q.fp8q_checkpoint_quantize(z, want_h, want_sf)
    for keep_d, keep_h, amax_on in ((True, True, True), (False, True, True), (False, False, True), (True, False, False)):
        bd, d = guarded((m, n), torch.bfloat16, dev)
        bq, q = guarded((m, n), torch.uint8, dev)
        bh, h = guarded((m, n), torch.uint8, dev)
        bs, sf = guarded((m, (n + 31) // 32), torch.uint8, dev)
        amax = torch.full((1,), 0.25, device=dev)
        fp8q.fp8q_matmul(A, B, d if keep_d else None, a_scale=s, bias=bias, act=1, residual=res, q=q, q_fmt=q_fmt, q_scale=qs,
                         amax=amax if amax_on else None, h=h if keep_h else None, h_sf=sf if keep_h else None)
        for t in (bd, bq, bh, bs):
            whole(t)
        assert torch.equal(q, want_q)
        if amax_on:
            assert torch.equal(amax, want_amax)
        if keep_d:
            assert torch.equal(d, y)
        if keep_h:
            assert torch.equal(h, want_h) and torch.equal(sf, want_sf)
    # the checkpoint alone, and amax alone
    h, sf = fp8q.checkpoint_empty(m, n)
    fp8q.fp8q_matmul(A, B, None, a_scale=s, bias=bias, act=1, h=h, h_sf=sf)
    assert torch.equal(h, want_h) and torch.equal(sf, want_sf)
    amax = torch.full((1,), 0.25, device=dev)
    fp8q.fp8q_matmul(A, B, None, a_scale=s, bias=bias, act=1, residual=res, amax=amax)
    assert torch.equal(amax, want_amax)


@pytest.mark.parametrize("m", [1, 40, 3000])
def test_gelu_over_its_range(dev, m):
    """The epilogue's GELU at every bf16, given by the bias of a product with an empty k: nothing else is rounded before it."""
    z = torch.arange(65536, dtype=torch.int32, device=dev).to(torch.int16).view(torch.bfloat16).float()
    z[:4096] = torch.linspace(-12, 12, 4096, device=dev)
    a, b = torch.empty((m, 0), dtype=torch.uint8, device=dev), torch.empty((65536, 0), dtype=torch.uint8, device=dev)
    d, y = torch.empty((m, 65536), device=dev), torch.empty((m, 65536), dtype=torch.bfloat16, device=dev)
    fp8q.fp8q_matmul(a, b, d, bias=z, act=1)
    fp8q.fp8q_matmul(a, b, y, bias=z, act=1)
    assert torch.equal(y[0], d[0].to(torch.bfloat16)) or torch.equal(y[0].isnan(), d[0].isnan())
    assert ((y == y[:1]) | y.isnan()).all() and ((d == d[:1]) | d.isnan()).all()
    x = z.double()
    want = torch.where(x < -30, torch.zeros_like(x), R.gelu(x))  # below, 0 in binary32 (and 1 + tanh 0 in 64 bits)
    want = torch.where(x > 30, x, want)
    # 1 + tanh loses what is left of it in 64 bits towards -6: there by exp
    u = -2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)
    want = torch.where((x < 0) & (x >= -30), x / (1 + torch.exp(u)), want)
    fine = torch.isfinite(z)
    rel = torch.where(x >= -5, 2.0 ** -18, 2.0 ** -16)
    bound = torch.where(x >= -10, rel * want.abs() + 2.0 ** -130, torch.full_like(x, 2.0 ** -100))
    assert ((d[0].double() - want).abs() <= bound)[fine].all()
    assert ((y[0].double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound) + 2.0 ** -134)[fine & (x.abs() < 2.0 ** 127)].all()
    assert d[0][z == float("inf")].eq(float("inf")).all() and d[0][z.isnan() | (z == -float("inf"))].isnan().all()


@pytest.mark.parametrize("m,n,k", EPILOGUE)
def test_checkpoint_beside_float32(dev, m, n, k):
    a, b = operands(dev, m, n, k, 8)
    A, B = stored(a, 0), stored(b, 0)
    bias, s = torch.randn(n, generator=gen(dev, 3), device=dev), torch.full((1,), 1.0 / k ** 0.5, device=dev)
    z = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    fp8q.fp8q_matmul(A, B, z, a_scale=s, bias=bias)
    want_h, want_sf = fp8q.checkpoint_empty(m, n)
    fp8q.fp8q_checkpoint_quantize(z, want_h, want_sf)
    for act in (0, 1):
        h, sf = fp8q.checkpoint_empty(m, n)
        d, ref = torch.empty((m, n), device=dev), torch.empty((m, n), device=dev)
        fp8q.fp8q_matmul(A, B, d, a_scale=s, bias=bias, act=act, h=h, h_sf=sf)
        fp8q.fp8q_matmul(A, B, ref, a_scale=s, bias=bias, act=act)
        assert torch.equal(h, want_h) and torch.equal(sf, want_sf) and torch.equal(d, ref)


@pytest.mark.parametrize("m,n,off", [(3, 200, 2), (130, 260, 1), (2600, 2304, 1), (2600, 2304, 2)])
def test_outputs_from_any_address(dev, m, n, off):
    k = 64
    a, b = operands(dev, m, n, k, 11)
    bias = torch.randn(n + off, generator=gen(dev, 1), device=dev)[off:]
    one = torch.ones(1, device=dev)
    want = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    want_q = torch.empty((m, n), dtype=torch.uint8, device=dev)
    want_h, want_sf = fp8q.checkpoint_empty(m, n)
    fp8q.fp8q_matmul(a, b, want, bias=bias.clone(), q=want_q, q_scale=one, h=want_h, h_sf=want_sf)
    room = [torch.full((m * n + 64,), CANARY, dtype=t, device=dev) for t in (torch.bfloat16, torch.uint8, torch.uint8)]
    d, q, h = (t[off: off + m * n].view(m, n) for t in room)
    sf = torch.empty_like(want_sf)
    fp8q.fp8q_matmul(a, b, d, bias=bias, q=q, q_scale=one, h=h, h_sf=sf)
    assert torch.equal(d, want) and torch.equal(q, want_q) and torch.equal(h, want_h) and torch.equal(sf, want_sf)
    for t in room:
        assert (t[:off] == CANARY).all() and (t[off + m * n:] == CANARY).all()


@pytest.mark.parametrize("m,n", [(1, 130), (40, 300), (300, 520), (2600, 2307)])
def test_empty_k(dev, m, n):
    a, b = torch.empty((m, 0), dtype=torch.uint8, device=dev), torch.empty((n, 0), dtype=torch.uint8, device=dev)
    bias = torch.randn(n, device=dev)
    res = torch.randn((m, n), device=dev)
    d = torch.full((m, n), 7.0, device=dev)
    fp8q.fp8q_matmul(a, b, d, bias=bias, residual=res)
    assert torch.equal(d, bias + res)
    fp8q.fp8q_matmul(a, b, d)
    assert not d.any()
    fp8q.fp8q_matmul(a[:0], b, d[:0])
    fp8q.fp8q_matmul(a, b[:0], d[:, :0].contiguous())


@pytest.mark.parametrize("ta,tb", [(0, 0), (1, 1)])
@pytest.mark.parametrize("m,n,k", [(20, 200, 300), (300, 200, 300), (2600, 2304, 288)])
def test_nan_and_infinity_stay_in_their_rows(dev, m, n, k, ta, tb):
    a, b = operands(dev, m, n, k, 21, 1, 0)
    a[2, k - 1], a[m - 1, 0], b[7, 5] = 0x7C, 0xFC, 0x7F  # infinities of e5m2, a NaN of e4m3
    va, vb = R.values(a, 1), R.values(b, 0)
    fine = torch.ones((m, n), dtype=torch.bool, device=dev)
    fine[2], fine[m - 1], fine[:, 7] = False, False, False
    d = torch.empty((m, n), device=dev)
    fp8q.fp8q_matmul(stored(a, ta), stored(b, tb), d, 1, 0, a_trans=ta, b_trans=tb)
    want = va.clone()
    want[2], want[m - 1] = 0, 0
    vb[7] = 0
    exact = want @ vb.t()
    assert torch.isfinite(d[fine]).all()
    assert ((d.double() - exact).abs() <= R.sum_bound(want, vb) + 2.0 ** -24 * exact.abs())[fine].all()
    assert not torch.isfinite(d[2]).any() and not torch.isfinite(d[m - 1]).any() and torch.isnan(d[:, 7]).all()
    # amax and codes of such rows, as the quantizer has them
    y, q, amax = torch.empty((m, n), dtype=torch.bfloat16, device=dev), torch.empty((m, n), dtype=torch.uint8, device=dev), torch.zeros(1, device=dev)
    one = torch.ones(1, device=dev)
    fp8q.fp8q_matmul(stored(a, ta), stored(b, tb), y, 1, 0, a_trans=ta, b_trans=tb, q=q, q_scale=one, amax=amax)
    q2 = torch.empty_like(q)
    fp8q.fp8q_quantize_amax(y, q2, 0, one, torch.zeros(1, device=dev))
    assert torch.equal(q, q2) and torch.isnan(amax).all()


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (48, 1024, 4096), (300, 520, 4096), (2600, 2304, 544)])
def test_same_bits_every_call_streams_and_graphs(dev, m, n, k):
    a, b = operands(dev, m, n, k, 31)
    bias = torch.randn(n, device=dev)
    qs = torch.full((1,), 0.3, device=dev)
    outs = []

    def call():
        d, q, amax = torch.empty((m, n), dtype=torch.bfloat16, device=dev), torch.empty((m, n), dtype=torch.uint8, device=dev), torch.zeros(1, device=dev)
        h, sf = fp8q.checkpoint_empty(m, n)
        fp8q.fp8q_matmul(a, b, d, bias=bias, act=1, q=q, q_scale=qs, amax=amax, h=h, h_sf=sf)
        return d, q, amax, h, sf

    first = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs.append(call())
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs.append(call())
    for _ in range(3):
        gr.replay()
    for _ in range(5):
        outs.append(call())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(o, first))


def test_slices_of_a_larger_matrix(dev):
    """Operands that are columns and rows of a larger one, as a fused projection's weight is cut."""
    g = gen(dev, 41)
    big_a, big_b = R.random_codes((70, 512), 0, g), R.random_codes((500, 512), 0, g)
    a, b = big_a[3:67, 128:368], big_b[100:441, 128:368]
    d = torch.empty((64, 341), device=dev)
    fp8q.fp8q_matmul(a, b, d)
    va, vb = R.values(a.contiguous(), 0), R.values(b.contiguous(), 0)
    check(d, va @ vb.t(), R.sum_bound(va, vb))
    fp8q.fp8q_matmul(big_a[:, 16:80], big_b[:70, 32:373], d, a_trans=True, b_trans=True)
    va, vb = R.values(big_a[:, 16:80].contiguous(), 0).t(), R.values(big_b[:70, 32:373].contiguous(), 0).t()
    check(d, va @ vb.t(), R.sum_bound(va, vb))


def test_refusals(dev):
    a, b = operands(dev, 8, 32, 64, 1)
    d = torch.empty((8, 32), device=dev)
    one = torch.ones(1, device=dev)
    q = torch.empty((8, 32), dtype=torch.uint8, device=dev)
    for bad in (dict(d=torch.empty((8, 31), device=dev)), dict(b=b[:, :48].contiguous()), dict(bias=torch.zeros(31, device=dev)),
                dict(residual=torch.zeros((8, 32), dtype=torch.bfloat16, device=dev)), dict(a=a.cpu()), dict(a=a.float()),
                dict(a=torch.empty((8, 72), dtype=torch.uint8, device=dev)[:, :64]), dict(a_scale=torch.ones(2, device=dev)),
                dict(d=torch.empty((32, 8), device=dev).t()), dict(a=a[0])):
        with pytest.raises(ValueError):
            fp8q.fp8q_matmul(**{**dict(a=a, b=b, d=d), **bad})
    for bad in (dict(d=d, q=q, q_scale=one), dict(d=None), dict(d=None, q=q), dict(d=d, a_fmt=2), dict(d=d, act=2), dict(d=d, amax=one),
                dict(d=None, h=q), dict(d=None, q=q, q_scale=one, q_fmt=3)):
        with pytest.raises(fp8q.Fp8qError) as e:
            fp8q.fp8q_matmul(a, b, **bad)
        assert e.value.status == 1
    with pytest.raises(fp8q.Fp8qError) as e:  # off a 16-byte boundary
        room = torch.empty(8 * 64 + 16, dtype=torch.uint8, device=dev)
        fp8q.fp8q_matmul(room[8: 8 + 8 * 64].view(8, 64), b, d)
    assert e.value.status == 2


@pytest.mark.parametrize("off", [0, 16])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(2600, 2320, 160), (5000, 3344, 96), (2600, 2304, 0), (257, 20016, 48)])
def test_residual_over_many_tiles(dev, m, n, k, out, off):
    """The residual's columns run ahead of the tiles: bit for bit the sum of it and of the call without it, in place and not, with
    rows that end within 32 columns, several tiles a CTA, and outputs on 16 and on 32 bytes."""
    g = gen(dev, m + n + k)
    a, b = R.random_codes((m, k), 0, g), R.random_codes((n, k), 0, g)
    A, B = stored(a, 0), stored(b, 0)
    bias = torch.randn(n, generator=g, device=dev)
    s = torch.full((1,), 0.1, device=dev)
    res = torch.randn((m, n), generator=g, device=dev).to(out)

    def room(dtype):
        size = torch.empty((), dtype=dtype).element_size()
        buf = torch.full((m * n * size + 256 + off,), CANARY, dtype=torch.uint8, device=dev)
        return buf, buf[128 + off: 128 + off + m * n * size].view(dtype).view(m, n)

    plain = torch.empty((m, n), device=dev)
    for act in (0, 1):
        fp8q.fp8q_matmul(A, B, plain, a_scale=s, bias=bias, act=act)
        want = (plain + res.float()).to(out)
        for same in (False, True):
            buf, d = room(out)
            if same:
                d.copy_(res)
            h, sf = fp8q.checkpoint_empty(m, n)
            fp8q.fp8q_matmul(A, B, d, a_scale=s, bias=bias, act=act, residual=d if same else res, h=h, h_sf=sf)
            assert torch.equal(d, want)
            assert (buf[: 128 + off] == CANARY).all() and (buf[-128:] == CANARY).all()
        h2, sf2 = fp8q.checkpoint_empty(m, n)
        fp8q.fp8q_matmul(A, B, None, a_scale=s, bias=bias, h=h2, h_sf=sf2)
        assert torch.equal(h, h2) and torch.equal(sf, sf2)
        if out == torch.bfloat16:
            buf, q = room(torch.uint8)
            q2, amax, amax2 = torch.empty((m, n), dtype=torch.uint8, device=dev), torch.zeros(1, device=dev), torch.zeros(1, device=dev)
            fp8q.fp8q_matmul(A, B, None, a_scale=s, bias=bias, act=act, residual=res, q=q, q_scale=s, amax=amax)
            fp8q.fp8q_quantize_amax(want, q2, 0, s, amax2)
            assert torch.equal(q, q2) and torch.equal(amax, amax2)
            assert (buf[: 128 + off] == CANARY).all() and (buf[-128:] == CANARY).all()
