"""The 4-bit operators and the residual norms run together, as a training step of a linear layer between two
norms uses them: norm -> codes -> product -> norm, and back through the second norm, the two products with the
transposed operands and the first norm.  Each stage is compared with its formula in float64 on what the stage
was given; and the same step on another stream, replayed from a graph, beside itself on two streams, and call
behind call without a wait between them gives the same bits."""
import os
import re

import numpy as np
import pytest
import torch

import fp4_reference as R
from conftest import ROOT
from gpu_helpers import bf16_bits_of
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp4 import product_bound
from test_gpu_residual_norm import check_forward, near_bf16, near_f32, reference_backward

pytestmark = pytest.mark.gpu
ALPHA, EPS = 0.7, 1e-6


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def inputs(rows, H, seed, fmt, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    f = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    d = {k: f(rows, H).bfloat16() for k in ("residual", "block", "d_out", "d_h2")}
    d["w"] = (f(H, H) * H ** -0.5).bfloat16()
    for k in ("post", "pre", "post2", "pre2"):
        d[k] = 1 + 0.2 * f(H)
    d["gate"], d["gate2"] = f(-(-rows // 50), H), f(-(-rows // 50), H).bfloat16()
    # one tensor scale for each operand, as a step with delayed scaling finds them
    d["scales"] = torch.tensor([5.0 / 2688, 0.2 / 2688, 0.05 / 2688], device=dev) if fmt == R.NVFP4 else None
    return d


def room(rows, H, fmt, dev):
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    f32 = lambda *s: torch.empty(s, device=dev)  # noqa: E731
    o = {k: bf(rows, H) for k in ("ro", "h", "y", "ro2", "h2", "dr2", "dy", "dh", "dr", "db")}
    o["dw"] = f32(H, H)
    for k in ("rstd_post", "rstd_pre", "rstd_post2", "rstd_pre2"):
        o[k] = f32(rows)
    for k in ("d_post", "d_pre", "d_post2", "d_pre2"):
        o[k] = f32(H)
    o["d_gate"], o["d_gate2"] = f32(-(-rows // 50), H), bf(-(-rows // 50), H)
    for k, (r, c) in {"x": (rows, H), "xt": (H, rows), "w": (H, H), "wt": (H, H), "g": (rows, H), "gt": (H, rows)}.items():
        o[k + "q"], o[k + "s"] = fp8q.fp4_empty(r, c, fmt, dev)
        o[k + "s"].fill_(0xEE)
    o["amax"] = torch.zeros(4, device=dev)
    o["space"] = torch.empty(fp8q.residual_norm_backward_workspace(rows, H, 50), dtype=torch.uint8, device=dev)
    return o


def step(d, o, fmt, stream=None, between=lambda: None):
    rows, H = d["residual"].shape
    sc = [None] * 3 if d["scales"] is None else [d["scales"][i: i + 1] for i in range(3)]
    amax = [o["amax"][i: i + 1] for i in range(4)]
    kw = {"stream": stream}
    norm = dict(rows_per_gate=50, alpha=ALPHA, eps=EPS, **kw)
    calls = [
        lambda: fp8q.fp8q_fp4_quantize_amax(d["w"], o["wq"], o["ws"], fmt, sc[1], amax[1], qt=o["wtq"], sft=o["wts"], **kw),
        lambda: fp8q.fp8q_residual_norm_quantize_amax(
            d["residual"], o["ro"], block=d["block"], post_weight=d["post"], gate=d["gate"], pre_weight=d["pre"], h=o["h"], q=o["xq"],
            sf=o["xs"], fmt=fmt, scale=sc[0], amax=amax[0], rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"], **norm),
        lambda: fp8q.fp8q_fp4_matmul(o["xq"], o["xs"], o["wq"], o["ws"], o["y"], H, fmt, sc[0], sc[1], **kw),
        lambda: fp8q.fp8q_residual_norm_quantize_amax(
            o["ro"], o["ro2"], block=o["y"], post_weight=d["post2"], gate=d["gate2"], pre_weight=d["pre2"], h=o["h2"], amax=amax[3],
            rstd_post=o["rstd_post2"], rstd_pre=o["rstd_pre2"], **norm),
        lambda: fp8q.fp8q_residual_norm_backward(
            d["d_out"], d["d_h2"], o["ro2"], o["rstd_pre2"], d["pre2"], o["dr2"], o["d_pre2"], block=o["y"], rstd_post=o["rstd_post2"],
            post_weight=d["post2"], gate=d["gate2"], rows_per_gate=50, alpha=ALPHA, d_block=o["dy"], d_post_weight=o["d_post2"],
            d_gate=o["d_gate2"], workspace=o["space"], **kw),
        lambda: fp8q.fp8q_fp4_quantize_amax(o["dy"], o["gq"], o["gs"], fmt, sc[2], amax[2], qt=o["gtq"], sft=o["gts"], **kw),
        lambda: fp8q.fp8q_fp4_quantize_amax(o["h"], None, None, fmt, sc[0], None, qt=o["xtq"], sft=o["xts"], **kw),
        lambda: fp8q.fp8q_fp4_matmul(o["gq"], o["gs"], o["wtq"], o["wts"], o["dh"], H, fmt, sc[2], sc[1], **kw),
        lambda: fp8q.fp8q_fp4_matmul(o["gtq"], o["gts"], o["xtq"], o["xts"], o["dw"], rows, fmt, sc[2], sc[0], **kw),
        lambda: fp8q.fp8q_residual_norm_backward(
            o["dr2"], o["dh"], o["ro"], o["rstd_pre"], d["pre"], o["dr"], o["d_pre"], block=d["block"], rstd_post=o["rstd_post"],
            post_weight=d["post"], gate=d["gate"], rows_per_gate=50, alpha=ALPHA, d_block=o["db"], d_post_weight=o["d_post"],
            d_gate=o["d_gate"], workspace=o["space"], **kw),
    ]
    for c in calls:
        c()
        between()


def same(a, b):
    for k in a:
        if k != "space":
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


SIZES = [(1, 64), (51, 528), (700, 1040), (2600, 1056)]


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("rows,H", SIZES)
def test_step(dev, rows, H, fmt):
    d, o = inputs(rows, H, rows + H, fmt, dev), room(rows, H, fmt, dev)
    step(d, o, fmt)
    sc = [None] * 3 if fmt == R.MXFP4 else [float(v) for v in d["scales"]]
    norm1 = {k: o[k] for k in ("ro", "h", "rstd_post", "rstd_pre")} | {"amax": o["amax"][0], "q": o["xq"], "sf": o["xs"], "scale": sc[0]}
    check_forward({k: d[k] for k in ("residual", "block", "post", "pre", "gate")}, norm1, rows, H, 50, ALPHA, EPS, fmt)
    norm2 = {"ro": o["ro2"], "h": o["h2"], "rstd_post": o["rstd_post2"], "rstd_pre": o["rstd_pre2"], "amax": o["amax"][3]}
    d2 = {"residual": o["ro"], "block": o["y"], "post": d["post2"], "pre": d["pre2"], "gate": d["gate2"]}
    check_forward(d2, norm2, rows, H, 50, ALPHA, EPS)

    v = {}
    for name, t, s in (("x", o["h"], sc[0]), ("w", d["w"], sc[1]), ("g", o["dy"], sc[2])):
        bits = bf16_bits_of(t).reshape(t.shape)
        for suffix, b in (("", bits), ("t", np.ascontiguousarray(bits.T))):
            codes, sf, nan = R.quantize(b, fmt, s)
            assert not nan.any()
            q, packed = R.pack(codes, sf)
            assert np.array_equal(o[name + suffix + "q"].cpu().numpy(), q), name + suffix
            assert np.array_equal(o[name + suffix + "s"].cpu().numpy(), packed), name + suffix
            v[name + suffix] = torch.from_numpy(R.values(codes, sf, fmt)).to(dev)
    assert float(o["amax"][1]) == float(d["w"].float().abs().max()) and float(o["amax"][2]) == float(o["dy"].float().abs().max())
    for name, a, b, k, i, j, eps in (("y", "x", "w", H, 0, 1, 2.0 ** -7), ("dh", "g", "wt", H, 2, 1, 2.0 ** -7),
                                     ("dw", "gt", "xt", rows, 2, 0, 2.0 ** -23)):
        alpha = 1.0 if fmt == R.MXFP4 else sc[i] * sc[j]
        want = (v[a] @ v[b].t()) * alpha
        off = (o[name].double() - want).abs()
        assert (off <= product_bound(v[a], v[b], want, k, alpha, eps)).all(), name

    for one, s, names in (
            (d2, {"ro": o["ro2"], "rstd_pre": o["rstd_pre2"], "rstd_post": o["rstd_post2"], "dro": d["d_out"], "dh": d["d_h2"]},
             {"d_residual": "dr2", "d_block": "dy", "d_pre_weight": "d_pre2", "d_post_weight": "d_post2", "d_gate": "d_gate2"}),
            (d, {"ro": o["ro"], "rstd_pre": o["rstd_pre"], "rstd_post": o["rstd_post"], "dro": o["dr2"], "dh": o["dh"]},
             {"d_residual": "dr", "d_block": "db", "d_pre_weight": "d_pre", "d_post_weight": "d_post", "d_gate": "d_gate"})):
        for name, (w, bound) in reference_backward(one, {**s, "block": True, "post": True}, rows, H, 50, ALPHA).items():
            got = o[names[name]]
            (near_bf16 if got.dtype == torch.bfloat16 else near_f32)(got, w, bound, names[name])


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("rows,H", SIZES)
def test_step_anywhere(dev, rows, H, fmt):
    """With a wait behind every call; without one, the buffers used again by the next step at once; on another
    stream; on two streams at a time; in a graph, behind a fill and beside work of a second stream."""
    ds = [inputs(rows, H, seed, fmt, dev) for seed in range(3)]
    want = []
    for d in ds:
        want.append(room(rows, H, fmt, dev))
        step(d, want[-1], fmt, between=torch.cuda.synchronize)

    o = room(rows, H, fmt, dev)
    for _ in range(4):
        for d, w in zip(ds, want):
            o["amax"].zero_()
            step(d, o, fmt)
            got = {k: t.clone() for k, t in o.items()}
            same(w, got)
    for _ in range(4):  # the same without a copy between the steps: only the last one's results are looked at
        for d in ds:
            o["amax"].zero_()
            step(d, o, fmt)
    same(want[2], o)

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    two = [room(rows, H, fmt, dev) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                two[i]["amax"].zero_()
            step(ds[i], two[i], fmt, stream=s)
    torch.cuda.synchronize()
    same(want[0], two[0])
    same(want[1], two[1])

    cur = {k: t.clone() if t is not None else None for k, t in ds[0].items()}
    graph, g = room(rows, H, fmt, dev), torch.cuda.CUDAGraph()
    other = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        graph["amax"].zero_()
        other.wait_stream(main)
        with torch.cuda.stream(other):
            step(cur, two[0], fmt)
        step(cur, graph, fmt)
        main.wait_stream(other)
        fp8q.fp8q_fp4_dequantize(graph["xq"], graph["xs"], two[1]["h"], fmt, None if cur["scales"] is None else cur["scales"][:1])
    for d, w in zip(ds, want):
        for k, t in d.items():
            if t is not None:
                cur[k].copy_(t)
        two[0]["amax"].zero_()
        g.replay()
        torch.cuda.synchronize()
        same(w, graph)
        same(w, two[0])
        y = torch.empty_like(two[1]["h"])
        fp8q.fp8q_fp4_dequantize(w["xq"], w["xs"], y, fmt, None if d["scales"] is None else d["scales"][:1])
        assert torch.equal(y, two[1]["h"])


def test_readme_example(dev):
    """The readme's second example, which goes on from its first."""
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)
    ns = {}
    for b in blocks:
        exec(compile(b, "readme example", "exec"), ns)
    torch.cuda.synchronize()
    assert float(ns["amax"]) > 1 and torch.isfinite(ns["y"]).all() and ns["y"].float().std() > 1
