"""The FP8 products, checkpoints and gradients run together, as training steps use them: an MLP (norm to codes -> up with
GELU, codes and checkpoint -> down into the residual stream, and back: quantized gradient, both gradient products of both
layers, the GELU's gradient from the checkpoint) and a layer of experts.  Each stage is compared with its formula in float64
on what the stage was given; and the same step on another stream, replayed from a graph, beside itself on two streams, and
call behind call without a wait between them gives the same bits."""
import pytest
import torch

import fp8_reference as R
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_fp8_matmul import check, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def mlp_inputs(rows, H, F, dev, seed=1):
    g = gen(dev, seed)
    f = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    d = {"residual": f(rows, H).bfloat16(), "block": f(rows, H).bfloat16(), "pre": 1 + 0.2 * f(H), "b1": 0.3 * f(F), "b2": f(H).bfloat16(),
         "dy": (1e-2 * f(rows, H)).bfloat16(), "w1": R.random_codes((F, H), 0, g, 1.0), "w2": R.random_codes((H, F), 0, g, 1.0)}
    for k, v in {"x": 5 / 448, "w1": H ** -0.5, "w2": F ** -0.5, "a": 6 / 448, "dy": 0.1 / 57344, "dh": 0.1 / 57344}.items():
        d["s_" + k] = torch.full((1,), v, device=dev)
    return d


def mlp_room(rows, H, F, dev):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device=dev)  # noqa: E731
    return {"ro": bf(rows, H), "x": u8(rows, H), "a": u8(rows, F), "h": u8(rows, F), "h_sf": u8(rows, (F + 31) // 32), "y": bf(rows, H),
            "dyq": u8(rows, H), "da": bf(rows, F), "dh": u8(rows, F), "db1": f32(F), "db2": f32(H), "dx": bf(rows, H), "dw1": f32(F, H),
            "dw2": f32(H, F), "amax": f32(4), "space": u8(max(1, fp8q.gelu_backward_workspace(rows, max(F, H))) + 4 * 4096 * (F + H))}


def mlp_step(d, o, stream=None, between=lambda: None):
    kw = {"stream": stream}
    am = [o["amax"][i: i + 1] for i in range(4)]
    E4, E5 = fp8q.E4M3FN, fp8q.E5M2
    calls = [
        lambda: fp8q.fp8q_residual_norm_quantize_amax(d["residual"], o["ro"], block=d["block"], pre_weight=d["pre"], q=o["x"], fmt=E4,
                                                      scale=d["s_x"], amax=am[0], **kw),
        lambda: fp8q.fp8q_matmul(o["x"], d["w1"], None, E4, E4, d["s_x"], d["s_w1"], bias=d["b1"], act=fp8q.ACT_GELU, q=o["a"], q_fmt=E4,
                                 q_scale=d["s_a"], amax=am[1], h=o["h"], h_sf=o["h_sf"], **kw),
        lambda: fp8q.fp8q_matmul(o["a"], d["w2"], o["y"], E4, E4, d["s_a"], d["s_w2"], bias=d["b2"], residual=o["ro"], **kw),
        lambda: fp8q.fp8q_gelu_backward_quantize_amax(d["dy"], None, None, o["dyq"], E5, d["s_dy"], am[2], d_bias=o["db2"], workspace=o["space"], **kw),
        lambda: fp8q.fp8q_matmul(o["dyq"], d["w2"], o["da"], E5, E4, d["s_dy"], d["s_w2"], b_trans=True, **kw),
        lambda: fp8q.fp8q_matmul(o["dyq"], o["a"], o["dw2"], E5, E4, d["s_dy"], d["s_a"], a_trans=True, b_trans=True, **kw),
        lambda: fp8q.fp8q_gelu_backward_quantize_amax(o["da"], o["h"], o["h_sf"], o["dh"], E5, d["s_dh"], am[3], d_bias=o["db1"],
                                                      workspace=o["space"], **kw),
        lambda: fp8q.fp8q_matmul(o["dh"], d["w1"], o["dx"], E5, E4, d["s_dh"], d["s_w1"], b_trans=True, **kw),
        lambda: fp8q.fp8q_matmul(o["dh"], o["x"], o["dw1"], E5, E4, d["s_dh"], d["s_x"], a_trans=True, b_trans=True, **kw),
    ]
    for c in calls:
        c()
        between()


def kept(o):
    return [v for k, v in o.items() if k != "space"]


@pytest.mark.parametrize("rows,H,F", [(5, 64, 272), (77, 256, 1040), (300, 1040, 2064), (2600, 768, 2304)])
def test_mlp_step(dev, rows, H, F):
    d, o = mlp_inputs(rows, H, F, dev), mlp_room(rows, H, F, dev)
    mlp_step(d, o, between=torch.cuda.synchronize)
    s = {k[2:]: float(v) for k, v in d.items() if k.startswith("s_")}
    x, w1, w2, a = R.values(o["x"], 0), R.values(d["w1"], 0), R.values(d["w2"], 0), R.values(o["a"], 0)
    # up: codes of a bf16 within its bound of the GELU are within half a step more
    z = x @ w1.t() * s["x"] * s["w1"] + d["b1"].double()
    off = R.sum_bound(x, w1) * s["x"] * s["w1"] + 2.0 ** -23 * z.abs()
    y = R.gelu(z)
    off_y = 1.13 * off + (2.0 ** -18 + 2.0 ** -8) * y.abs()
    q = y.clamp(-448 * s["a"], 448 * s["a"])
    assert ((a * s["a"] - q).abs() <= off_y + 2.0 ** -4 * (q.abs() + off_y) + 2.0 ** -10 * s["a"]).all()
    h = torch.empty((rows, F), dtype=torch.bfloat16, device=dev)
    fp8q.fp8q_checkpoint_dequantize(o["h"], o["h_sf"], h)
    step = torch.exp2(o["h_sf"].double() - 127 - 10).repeat_interleave(32, 1)[:, :F]
    off_h = off + 2.0 ** -8 * (z.abs() + off)
    assert ((h.double() - z).abs() <= off_h + torch.maximum(2.0 ** -4 * (z.abs() + off_h), step)).all()
    # down
    want = a @ w2.t() * s["a"] * s["w2"] + d["b2"].double() + o["ro"].double()
    check(o["y"], want, R.sum_bound(a, w2) * s["a"] * s["w2"] + 2.0 ** -22 * (want.abs() + o["ro"].double().abs()))
    # back
    want_q = torch.empty_like(o["dyq"])
    fp8q.fp8q_quantize_amax(d["dy"], want_q, 1, d["s_dy"], torch.zeros(1, device=dev))
    assert torch.equal(o["dyq"], want_q)
    assert ((o["db2"].double() - d["dy"].double().sum(0)).abs() <= (rows + 2) * 2.0 ** -24 * d["dy"].double().abs().sum(0)).all()
    dy, dh = R.values(o["dyq"], 1), R.values(o["dh"], 1)
    check(o["da"], dy @ w2 * s["dy"] * s["w2"], R.sum_bound(dy, w2.t()) * s["dy"] * s["w2"])
    check(o["dw2"], dy.t() @ a * s["dy"] * s["a"], R.sum_bound(dy.t(), a.t()) * s["dy"] * s["a"])
    g = o["da"].double() * R.gelu_slope(h)
    off = o["da"].double().abs() * 2.0 ** -19 * (1 + h.double().abs().clamp(max=10)) + 2.0 ** -24 * g.abs()
    assert ((o["db1"].double() - g.sum(0)).abs() <= off.sum(0) + (rows + 2) * 2.0 ** -24 * g.abs().sum(0)).all()
    off = off + 2.0 ** -8 * (g.abs() + off)
    q = g.clamp(-57344 * s["dh"], 57344 * s["dh"])
    assert ((dh * s["dh"] - q).abs() <= off + 2.0 ** -3 * (q.abs() + off) + 2.0 ** -17 * s["dh"]).all()
    check(o["dx"], dh @ w1 * s["dh"] * s["w1"], R.sum_bound(dh, w1.t()) * s["dh"] * s["w1"])
    check(o["dw1"], dh.t() @ x * s["dh"] * s["x"], R.sum_bound(dh.t(), x.t()) * s["dh"] * s["x"])


@pytest.mark.parametrize("rows,H,F", [(5, 64, 272), (300, 1040, 2064), (2600, 768, 2304)])
def test_mlp_step_on_streams_in_graphs_and_without_waits(dev, rows, H, F):
    d, first = mlp_inputs(rows, H, F, dev), mlp_room(rows, H, F, dev)
    mlp_step(d, first, between=torch.cuda.synchronize)
    plain = mlp_room(rows, H, F, dev)
    mlp_step(d, plain)
    outs = [plain]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (a, b):  # side by side
        outs.append(mlp_room(rows, H, F, dev))
    torch.cuda.synchronize()
    for s, o in zip((a, b), outs[1:]):
        mlp_step(d, o, stream=s)
    torch.cuda.synchronize()
    o = mlp_room(rows, H, F, dev)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        mlp_step(d, o)
    for _ in range(3):
        gr.replay()
    outs.append(o)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(u, v) for u, v in zip(kept(o), kept(first)))


@pytest.mark.parametrize("rows,e,H,F", [(9, 4, 64, 272), (300, 7, 272, 528), (2600, 5, 528, 1040)])
def test_experts_step(dev, rows, e, H, F):
    """Up with GELU, codes and checkpoint, down, and the gradients back to the experts' inputs and weights."""
    g = gen(dev, rows)
    cut = torch.randint(0, rows + 1, (e - 1,), generator=g, device=dev).sort().values
    cut[e // 2 - 1] = cut[e // 2]  # an expert without rows
    off = torch.cat((torch.zeros(1, device=dev), cut, torch.full((1,), rows, device=dev))).to(torch.int32)
    f = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    x, w1, w2 = R.random_codes((rows, H), 0, g, 1.0), R.random_codes((e, F, H), 0, g, 1.0), R.random_codes((e, H, F), 0, g, 1.0)
    b1, dy = 0.3 * f(e, F), R.random_codes((rows, H), 1, g, 1.0)
    s1, s2, sa = (torch.full((1,), v, device=dev) for v in (H ** -0.5, F ** -0.5, 6 / 448))

    def step():
        a, y, da, dx = torch.empty((rows, F), dtype=torch.uint8, device=dev), bf(rows, H), bf(rows, F), bf(rows, H)
        h, h_sf = fp8q.checkpoint_empty(rows, F)
        dh, amax = torch.empty((rows, F), dtype=torch.uint8, device=dev), torch.zeros(2, device=dev)
        dw1, dw2 = torch.empty((e, F, H), device=dev), bf(e, H, F)
        fp8q.fp8q_grouped_matmul(x, w1, off, None, 0, 0, s1, None, bias=b1, act=1, q=a, q_scale=sa, amax=amax[:1], h=h, h_sf=h_sf)
        fp8q.fp8q_grouped_matmul(a, w2, off, y, 0, 0, sa, s2)
        fp8q.fp8q_grouped_matmul(dy, w2, off, da, 1, 0, None, s2, b_trans=True)
        fp8q.fp8q_grouped_weight_gradient(dy, a, off, dw2, 1, 0, None, sa)
        fp8q.fp8q_gelu_backward_quantize_amax(da, h, h_sf, dh, 1, s1, amax[1:])
        fp8q.fp8q_grouped_matmul(dh, w1, off, dx, 1, 0, s1, s1, b_trans=True)
        fp8q.fp8q_grouped_weight_gradient(dh, x, off, dw1, 1, 0, s1, None)
        return a, y, da, dx, dh, amax, dw1, dw2, h, h_sf

    out = step()
    a, y, da, dx, dh, amax, dw1, dw2, h, h_sf = out
    va, vx, vy, vh = R.values(a, 0), R.values(x, 0), R.values(dy, 1), R.values(dh, 1)
    f1, f2, fa = float(s1), float(s2), float(sa)
    for i in range(e):
        lo, hi = int(off[i]), int(off[i + 1])
        v1, v2, r = R.values(w1[i], 0), R.values(w2[i], 0), slice(lo, hi)
        if lo < hi:
            check(y[r], va[r] @ v2.t() * fa * f2, R.sum_bound(va[r], v2) * fa * f2)
            check(da[r], vy[r] @ v2 * f2, R.sum_bound(vy[r], v2.t()) * f2)
            check(dx[r], vh[r] @ v1 * f1 * f1, R.sum_bound(vh[r], v1.t()) * f1 * f1)
            z = vx[r] @ v1.t() * f1 + b1[i].double()
            bound = 1.13 * (R.sum_bound(vx[r], v1) * f1 + 2.0 ** -23 * z.abs()) + (2.0 ** -18 + 2.0 ** -8) * R.gelu(z).abs()
            q = R.gelu(z).clamp(-448 * fa, 448 * fa)
            assert ((va[r] * fa - q).abs() <= bound + 2.0 ** -4 * (q.abs() + bound) + 2.0 ** -10 * fa).all()
        check(dw2[i], vy[r].t() @ va[r] * fa, R.sum_bound(vy[r].t(), va[r].t()) * fa)
        check(dw1[i], vh[r].t() @ vx[r] * f1, R.sum_bound(vh[r].t(), vx[r].t()) * f1)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        again = step()
    gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(out, again))


def test_readme_example():
    """The readme's MLP runs as written, behind the examples before it, and moves what it says."""
    import os
    import re

    from conftest import ROOT
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    ns = {}
    for b in blocks[:3]:
        exec(compile(b, "readme example", "exec"), ns)
    torch.cuda.synchronize()
    x, w1, s = R.values(ns["x8"], 0), R.values(ns["w1"], 0), 8.0 / 448
    z = x @ w1.t() * s * s
    a = R.values(ns["a8"], 0) * s
    want = R.gelu(z).clamp(-8, 8)
    assert ((a - want).abs() <= 0.07 * want.abs() + 2.0 ** -9 * s + 2.0 ** -16).all()  # half steps of bf16 and of e4m3
    d1 = R.values(ns["d1"], 1)
    check(ns["dw1"], d1.t() @ x * 1e-6 * s, (R.sum_bound(d1.t(), x.t()) + (d1.t() @ x).abs() * 2.0 ** -23) * 1e-6 * s)
    assert ns["db1"].any() and torch.isfinite(ns["dw2"]).all() and ns["dw2"].any() and ns["out"].any()
