"""The 4-bit and residual-norm calls are one kernel launch each, the gradients two where they sum over rows, and an
empty sum one fill; their first use in a process may be captured; and what a call has captured goes on with the inputs
of each replay."""
import os
import subprocess
import sys

import pytest
import torch

import fp4_reference as R
from conftest import ROOT
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_launch_count import _graph_nodes

pytestmark = pytest.mark.gpu


def calls(dev, rows, H, n, fmt):
    bf = lambda *s: torch.randn(s, device=dev).bfloat16()  # noqa: E731
    f32 = lambda *s: torch.ones(s, device=dev)  # noqa: E731
    x, block, dh, dr, db, h = (bf(rows, H) for _ in range(6))
    q, sf = fp8q.fp4_empty(rows, H, fmt)
    qt, sft = fp8q.fp4_empty(H, rows, fmt)
    w = fp8q.fp4_empty(n, H, fmt)
    fp8q.fp8q_fp4_quantize_amax(bf(n, H), *w, fmt)
    y, yf, amax, q8 = bf(rows, n), f32(rows, n), f32(1), torch.empty((rows, H), dtype=torch.uint8, device=dev)
    post, pre, gate, gate1, r1, r2 = f32(H), f32(H), f32(-(-rows // 3), H), bf(rows, H), f32(rows), f32(rows)
    space = torch.empty(fp8q.residual_norm_backward_workspace(rows, H, 3), dtype=torch.uint8, device=dev)
    none, none_w = fp8q.fp4_empty(rows, 0, fmt), fp8q.fp4_empty(n, 0, fmt)
    edge = dict(block=block, post_weight=post, pre_weight=pre, rstd_post=r1, rstd_pre=r2)
    back = dict(block=block, rstd_post=r1, post_weight=post, d_block=db)
    return {
        "quantize": (lambda: fp8q.fp8q_fp4_quantize_amax(x, q, sf, fmt, None, amax), 1, 1),
        "quantize both": (lambda: fp8q.fp8q_fp4_quantize_amax(x, q, sf, fmt, None, amax, qt=qt, sft=sft), 1, 1),
        "quantize transposed": (lambda: fp8q.fp8q_fp4_quantize_amax(x, None, None, fmt, qt=qt, sft=sft), 1, 1),
        "dequantize": (lambda: fp8q.fp8q_fp4_dequantize(q, sf, h, fmt), 1, 1),
        "product": (lambda: fp8q.fp8q_fp4_matmul(q, sf, *w, y, H, fmt), 1, 1),
        "product, float32": (lambda: fp8q.fp8q_fp4_matmul(q, sf, *w, yf, H, fmt), 1, 1),
        "product of nothing": (lambda: fp8q.fp8q_fp4_matmul(*none, *none_w, y, 0, fmt), 0, 1),
        "norm": (lambda: fp8q.fp8q_residual_norm_quantize_amax(x, dr, gate=gate, rows_per_gate=3, q=q, sf=sf, fmt=fmt, amax=amax, **edge), 1, 1),
        "norm, a gate a token": (lambda: fp8q.fp8q_residual_norm_quantize_amax(x, dr, gate=gate1, rows_per_gate=1, q=q8, fmt=0, scale=amax, **edge),
                                 1, 1),
        "gradients of rows": (lambda: fp8q.fp8q_residual_norm_backward(x, dh, x, r2, pre, dr, None, **back), 1, 1),
        "gradients of rows, a gate a token": (lambda: fp8q.fp8q_residual_norm_backward(x, dh, x, r2, pre, dr, None, gate=gate1, rows_per_gate=1,
                                                                                       d_gate=h, **back), 1, 1),
        "gradients": (lambda: fp8q.fp8q_residual_norm_backward(x, dh, x, r2, pre, dr, torch.empty_like(pre), gate=gate, rows_per_gate=3,
                                                               d_gate=torch.empty_like(gate), d_post_weight=torch.empty_like(post),
                                                               workspace=space, **back), 2, 2),
    }


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("rows,H,n", [(1, 4096, 512), (70, 2064, 200), (2560, 1056, 2304), (33, 16384, 64)])
def test_launches(rows, H, n, fmt):
    dev = torch.device("cuda:0")
    s = torch.cuda.Stream()
    todo = calls(dev, rows, H, n, fmt)
    torch.cuda.synchronize()
    for name, (fn, kernels, nodes) in todo.items():
        assert _graph_nodes(fn, s) == (kernels, nodes), name


FIRST = r"""
import torch
from quantize_amax_scaling_gb300 import fp8q
dev, fmt = torch.device("cuda:0"), %d
rows, H, n = %d, %d, %d
g = torch.Generator(device=dev)
g.manual_seed(5)
f = lambda *s: torch.randn(s, generator=g, device=dev)
res, block, w, pre, post, gate = f(rows, H).bfloat16(), f(rows, H).bfloat16(), f(n, H).bfloat16(), f(H), f(H), f(1, H)
dro, dh = f(rows, H).bfloat16(), f(rows, H).bfloat16()

def room():
    o = {k: torch.zeros(rows, H, dtype=torch.bfloat16, device=dev) for k in ("ro", "h", "dr", "db")}
    o |= {k: torch.zeros(H, device=dev) for k in ("dpre", "dpost")} | {k: torch.zeros(rows, device=dev) for k in ("r1", "r2")}
    o["dg"], o["y"], o["amax"] = torch.zeros(1, H, device=dev), torch.zeros(rows, n, device=dev), torch.zeros(1, device=dev)
    for k, a, b in (("x", rows, H), ("w", n, H), ("t", H, n)):
        o[k + "q"] = torch.zeros(a, fp8q.fp4_row_bytes(b), dtype=torch.uint8, device=dev)
        o[k + "s"] = torch.zeros(fp8q.fp4_scale_bytes(a, b, fmt), dtype=torch.uint8, device=dev)
    o["space"] = torch.zeros(4 << 24, dtype=torch.uint8, device=dev)
    return o

def step(o):
    fp8q.fp8q_fp4_quantize_amax(w, o["wq"], o["ws"], fmt, qt=o["tq"], sft=o["ts"])
    fp8q.fp8q_residual_norm_quantize_amax(res, o["ro"], block=block, post_weight=post, gate=gate, rows_per_gate=rows, pre_weight=pre, h=o["h"],
                                          q=o["xq"], sf=o["xs"], fmt=fmt, amax=o["amax"], rstd_post=o["r1"], rstd_pre=o["r2"])
    fp8q.fp8q_fp4_matmul(o["xq"], o["xs"], o["wq"], o["ws"], o["y"], H, fmt)
    fp8q.fp8q_fp4_dequantize(o["xq"], o["xs"], o["h"], fmt)
    fp8q.fp8q_residual_norm_backward(dro, dh, o["ro"], o["r2"], pre, o["dr"], o["dpre"], block=block, rstd_post=o["r1"], post_weight=post, gate=gate,
                                     rows_per_gate=rows, d_block=o["db"], d_post_weight=o["dpost"], d_gate=o["dg"], workspace=o["space"])

first, eager = room(), room()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr, stream=torch.cuda.Stream()):
    step(first)
gr.replay()
torch.cuda.synchronize()
step(eager)
torch.cuda.synchronize()
assert eager["y"].any() and all(torch.equal(first[k], eager[k]) for k in eager if k != "space")
gr.replay()  # amax holds the same maximum, everything else is written anew
torch.cuda.synchronize()
assert all(torch.equal(first[k], eager[k]) for k in eager if k != "space")
print("OK")
"""


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
@pytest.mark.parametrize("rows,H,n", [(3, 1040, 200), (2560, 1056, 2304), (40, 12304, 130)])
def test_first_call_inside_graph_capture(rows, H, n, fmt):
    """In a fresh process: shared-memory limits, tensor maps and the SM count are asked for within the capture."""
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", FIRST % (fmt, rows, H, n)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout + r.stderr
