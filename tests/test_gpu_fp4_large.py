"""The 4-bit operators and the residual norms where they could go wrong by size alone: more than 2^32 elements,
whose last rows have to come out as those rows by themselves do, and none at all."""
import pytest
import torch

import fp4_reference as R
from quantize_amax_scaling_gb300 import fp8q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if torch.cuda.get_device_properties(0).total_memory < 150 << 30:
        pytest.skip("needs 150 GB of device memory")
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def big(rows, cols, seed, dev):
    """[rows, cols] bf16, every row and column of its own size."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    return torch.mul(torch.randn((rows, 1), generator=g, device=dev).bfloat16(), torch.randn((1, cols), generator=g, device=dev).bfloat16(), out=x)


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("rows,cols", [(131205, 32768), (131205, 32770)])
def test_quantize_and_back(dev, rows, cols, fmt):
    x = big(rows, cols, 1, dev)
    first = rows // 128 * 128 - 128  # the last whole tile of rows and the part behind it
    tail = x[first:]
    whole, one = [], []
    for t, to in ((x, whole), (tail, one)):
        r = t.shape[0]
        to += [*fp8q.fp4_empty(r, cols, fmt, dev), *fp8q.fp4_empty(cols, r, fmt, dev), torch.zeros(1, device=dev)]
        to[1].zero_(), to[3].zero_()
        fp8q.fp8q_fp4_quantize_amax(t, to[0], to[1], fmt, None, to[4], qt=to[2], sft=to[3])
        y = torch.empty_like(t)
        fp8q.fp8q_fp4_dequantize(to[0], to[1], y, fmt)
        to.append(y)
    across = -(-cols // (4 * R.BLOCK[fmt]))
    assert torch.equal(whole[0][first:], one[0])
    assert torch.equal(whole[1].view(-1, across, 512)[first // 128:], one[1].view(-1, across, 512))
    assert torch.equal(whole[2][:, first // 2:], one[2])
    assert torch.equal(whole[3].view(-(-cols // 128), -1, 512)[:, first // (4 * R.BLOCK[fmt]):], one[3].view(-(-cols // 128), -1, 512))
    assert torch.equal(whole[5][first:], one[5])
    assert float(whole[4]) == max(float(x[i:i + 8192].abs().max()) for i in range(0, rows, 8192))


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 65536), (torch.bfloat16, 65537), (torch.float32, 65536)])
def test_matmul(dev, dtype, n):
    """Sums that binary32 holds exactly, so that the tail's own product is the same whatever kernel takes it."""
    m, k, fmt = 65536 + 300, 96, R.NVFP4
    g = torch.Generator(device=dev)
    g.manual_seed(n)
    op = []
    for r in (m, n):
        q, s = fp8q.fp4_empty(r, k, fmt, dev)
        q.random_(0, 256, generator=g)
        op += [q, s.fill_(0x38)]
    d = torch.empty((m, n), dtype=dtype, device=dev)
    fp8q.fp8q_fp4_matmul(*op, d, k, fmt)
    first = m // 128 * 128 - 128
    tail = torch.empty((m - first, n), dtype=dtype, device=dev)
    fp8q.fp8q_fp4_matmul(op[0][first:], op[1].view(-1, 2 * 512)[first // 128:].reshape(-1), *op[2:], tail, k, fmt)
    assert torch.equal(d[first:], tail)
    head = torch.empty((200, n), dtype=dtype, device=dev)
    fp8q.fp8q_fp4_matmul(op[0][:200], op[1][:2 * 1024], *op[2:], head, k, fmt)
    assert torch.equal(d[:200], head)


@pytest.mark.parametrize("fmt", [0, R.NVFP4])
@pytest.mark.parametrize("rows,H", [(131100, 32768), (1049000, 4096)])
def test_residual_norm(dev, rows, H, fmt):
    per = 1024
    g = torch.Generator(device=dev)
    g.manual_seed(rows)
    f = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    res, block, post, pre, gate = big(rows, H, 3, dev), big(rows, H, 4, dev), 1 + 0.1 * f(H), 1 + 0.1 * f(H), f(-(-rows // per), H)
    dro, dh = big(rows, H, 5, dev), big(rows, H, 6, dev)
    scale = torch.full((1,), 0.01, device=dev)
    first = rows // per * per - per  # rows and gate rows of the tail

    def run(at):
        n = rows - at
        o = {"ro": torch.empty_like(res[at:]), "rpost": torch.empty(n, device=dev), "rpre": torch.empty(n, device=dev)}
        if fmt == R.NVFP4:
            o["q"], o["sf"] = fp8q.fp4_empty(n, H, fmt, dev)
            o["sf"].zero_()
        else:
            o["q"] = torch.empty((n, H), dtype=torch.uint8, device=dev)
        fp8q.fp8q_residual_norm_quantize_amax(res[at:], o["ro"], block=block[at:], post_weight=post, gate=gate[at // per:], rows_per_gate=per,
                                              alpha=0.5, pre_weight=pre, q=o["q"], sf=o.get("sf"), fmt=fmt, scale=scale, rstd_post=o["rpost"],
                                              rstd_pre=o["rpre"])
        o["dr"], o["db"] = torch.empty_like(o["ro"]), torch.empty_like(o["ro"])
        sums = [torch.empty(H, device=dev), torch.empty(H, device=dev), torch.empty_like(gate[at // per:])]
        room = torch.empty(fp8q.residual_norm_backward_workspace(n, H, per), dtype=torch.uint8, device=dev)
        fp8q.fp8q_residual_norm_backward(dro[at:], dh[at:], o["ro"], o["rpre"], pre, o["dr"], sums[0], block=block[at:], rstd_post=o["rpost"],
                                         post_weight=post, gate=gate[at // per:], rows_per_gate=per, alpha=0.5, d_block=o["db"],
                                         d_post_weight=sums[1], d_gate=sums[2], workspace=room)
        for s in sums:
            assert torch.isfinite(s).all()
        return o

    whole, tail = run(0), run(first)
    for k, t in tail.items():
        w = whole[k].view(-1, 512 * (-(-H // 64)))[first // 128:].reshape(-1) if k == "sf" else whole[k][first:]
        assert torch.equal(w, t), k


def test_nothing_at_all(dev):
    """No rows: the sums over them are zeros, and nothing else is written.  An empty k: the product is zeros."""
    H = 272
    e = torch.empty((0, H), dtype=torch.bfloat16, device=dev)
    z = torch.empty(0, device=dev)
    w = torch.ones(H, device=dev)
    dpre, dpost = torch.full((H,), 7.0, device=dev), torch.full((H + 4,), 7.0, device=dev)
    gate = torch.empty((0, H), device=dev)
    fp8q.fp8q_residual_norm_quantize_amax(e, e, block=e, post_weight=w, gate=gate, rows_per_gate=2, pre_weight=w, h=e)
    fp8q.fp8q_residual_norm_backward(e, e, e, z, w, e, dpre, block=e, rstd_post=z, post_weight=w, gate=gate, rows_per_gate=2, d_block=e,
                                     d_post_weight=dpost[:H], d_gate=gate, workspace=torch.empty(0, dtype=torch.uint8, device=dev))
    assert not dpre.any() and not dpost[:H].any() and (dpost[H:] == 7).all()
    for dtype in (torch.bfloat16, torch.float32):
        for m, n in ((3, 5), (300, 129)):
            d = torch.full((m * n + 8,), 7.0, dtype=dtype, device=dev)
            fp8q.fp8q_fp4_matmul(*fp8q.fp4_empty(m, 0, R.NVFP4, dev), *fp8q.fp4_empty(n, 0, R.NVFP4, dev), d[:m * n].view(m, n), 0, R.NVFP4)
            assert not d[:m * n].any() and (d[m * n:] == 7).all()


def test_handed_from_stream_to_stream(dev):
    """Quantize on one stream, multiply on another, events between them, one set of buffers."""
    fmt, m, n, k = R.NVFP4, 300, 520, 1040
    xs = [big(m, k, i, dev) for i in range(4)]
    w = fp8q.fp4_empty(n, k, fmt, dev)
    fp8q.fp8q_fp4_quantize_amax(big(n, k, 9, dev), *w, fmt)
    p, want = fp8q.fp4_empty(m, k, fmt, dev), []
    for x in xs:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
        fp8q.fp8q_fp4_quantize_amax(x, *p, fmt)
        torch.cuda.synchronize()
        fp8q.fp8q_fp4_matmul(*p, *w, d, k, fmt)
        torch.cuda.synchronize()
        want.append(d)
    a, b = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
    got = [torch.empty_like(d) for d in want * 8]
    torch.cuda.synchronize()
    for i, d in enumerate(got):
        fp8q.fp8q_fp4_quantize_amax(xs[i % 4], *p, fmt, stream=a)
        b.wait_stream(a)
        fp8q.fp8q_fp4_matmul(*p, *w, d, k, fmt, stream=b)
        a.wait_stream(b)
    torch.cuda.synchronize()
    for i, d in enumerate(got):
        assert torch.equal(d, want[i % 4]), i
