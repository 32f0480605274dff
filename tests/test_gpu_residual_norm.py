"""The RMS norms after and before a block with gate, residual scale and quantization, forward and
backward, against their formulas in float64.

Tolerances, with u = 2^-24.  A row's sum of H terms is taken 16 or 32 terms a thread, over 5 warp steps and
at most 32 warps or 8 warps and 8 slices, so no term passes through more than 70 additions, each product
adds one rounding: a mean is off by at most 72 u of the mean of the absolute terms, 1 / sqrt by half that and 3 u more
(40 u).  Every other step adds u.  A bf16 output is the rounding of a value within the bound of the true one."""
import numpy as np
import pytest
import torch

import fp4_reference as R
import oracle
from gpu_helpers import assert_codes_equal, bf16_bits_of
from quantize_amax_scaling_gb300 import fp8q

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def near_bf16(got, want, bound, what):
    """got (bf16) is the rounding of some value within `bound` of `want` (float64)."""
    lo, hi = (want - bound).float(), (want + bound).float()
    # one step outward for the conversion to float, then round: rounding is monotonic
    lo = torch.nextafter(lo, torch.full_like(lo, -float("inf"))).to(torch.bfloat16).double()
    hi = torch.nextafter(hi, torch.full_like(hi, float("inf"))).to(torch.bfloat16).double()
    g = got.double()
    bad = ~((g >= lo) & (g <= hi))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def near_f32(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound + 2.0 ** -23 * want.abs())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / (bound + 1e-300)).max()):.3g} bounds"


def make(rows, H, per, gate, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    f = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    groups = -(-rows // per) if per else 0
    d = {"residual": (2 * f(rows, H)).bfloat16(), "block": (f(rows, H) * torch.exp2(4 * f(rows, 1))).bfloat16(),
         "post": 1 + 0.3 * f(H), "pre": 1 + 0.3 * f(H), "gate": None}
    if gate:
        d["gate"] = f(groups, H).to(torch.float32 if gate == "f32" else torch.bfloat16)
    return d


def gate_rows(gate, rows, per):
    return gate.double()[torch.arange(rows, device=gate.device) // per] if gate is not None else 1.0


def forward(d, rows, H, per, alpha, eps, *, fmt=0, scale=0.01, block=True, post=True, pre=True, want_h=True, want_q=True, dev=None):
    o = {"ro": torch.full((rows, H), 7.0, dtype=torch.bfloat16, device=dev)}
    kw = {}
    if pre:
        o["amax"] = torch.zeros(1, device=dev)
        if want_h:
            o["h"] = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device=dev)
        if want_q:
            o["scale"] = None if fmt == R.MXFP4 else torch.full((1,), scale, device=dev)
            if fmt in (R.MXFP4, R.NVFP4):
                o["q"], o["sf"] = fp8q.fp4_empty(rows, H, fmt, dev)
                o["sf"].fill_(0xEE)
            else:
                o["q"] = torch.empty((rows, H), dtype=torch.uint8, device=dev)
        o["rstd_pre"] = torch.empty(rows, device=dev)
        kw = dict(pre_weight=d["pre"], h=o.get("h"), q=o.get("q"), sf=o.get("sf"), fmt=fmt, scale=o.get("scale"), amax=o["amax"],
                  rstd_pre=o["rstd_pre"])
    if block:
        o["rstd_post"] = torch.empty(rows, device=dev) if post else None
        kw |= dict(block=d["block"], post_weight=d["post"] if post else None, gate=d["gate"], rows_per_gate=per, alpha=alpha,
                   rstd_post=o["rstd_post"])
    fp8q.fp8q_residual_norm_quantize_amax(d["residual"], o["ro"], eps=eps, **kw)
    return o


def check_forward(d, o, rows, H, per, alpha, eps, fmt=0, block=True, post=True):
    r, b = d["residual"].double(), d["block"].double()
    if block:
        y = b
        if post:
            rstd = 1 / torch.sqrt(b.square().mean(1) + eps)
            near_f32(o["rstd_post"], rstd, 40 * U * rstd, "rstd_post")
            y = b * rstd[:, None] * d["post"].double()
        t = alpha * gate_rows(d["gate"], rows, per) * y
        near_bf16(o["ro"], r + t, 48 * U * t.abs() + 2 * U * (r + t).abs(), "residual_out")
    else:
        assert torch.equal(o["ro"], d["residual"])
    if "rstd_pre" not in o:
        return
    v = o["ro"].double()
    rstd = 1 / torch.sqrt(v.square().mean(1) + eps)
    near_f32(o["rstd_pre"], rstd, 40 * U * rstd, "rstd_pre")
    h = v * rstd[:, None] * d["pre"].double()
    if "h" in o:
        near_bf16(o["h"], h, 44 * U * h.abs() + 2.0 ** -133, "h")
        hb = bf16_bits_of(o["h"])
        assert float(o["amax"]) == float(o["h"].float().abs().max())
        if "q" in o:
            if fmt in (R.MXFP4, R.NVFP4):
                codes, sf, _ = R.quantize(hb.reshape(rows, H), fmt, None if o["scale"] is None else float(o["scale"]))
                q, s = R.pack(codes, sf)
                assert np.array_equal(o["q"].cpu().numpy(), q) and np.array_equal(o["sf"].cpu().numpy(), s)
            else:
                rq, _ = oracle.quantize_amax(hb, fmt, np.float32(float(o["scale"])))
                assert_codes_equal(o["q"].cpu().numpy(), rq, fmt)


SHAPES = [(1, 16), (3, 48), (5, 256), (9, 512), (2, 528), (130, 80), (67, 1040), (129, 2048), (33, 2064), (1, 4096), (20, 4112), (7, 8192),
          (5, 12304), (3, 16384), (2, 16400), (2, 32768), (1000, 64)]


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
@pytest.mark.parametrize("rows,H", SHAPES)
def test_forward(dev, rows, H, fmt):
    per = {0: 1, 1: rows, 2: max(1, rows // 3), 3: 2}[fmt]
    d = make(rows, H, per, "bf16" if fmt % 2 else "f32", rows + H, dev)
    o = forward(d, rows, H, per, 0.7, 1e-6, fmt=fmt, dev=dev)
    check_forward(d, o, rows, H, per, 0.7, 1e-6, fmt)
    # without h, in place: the same codes, residual and amax
    e = dict(d, residual=d["residual"].clone())
    q = torch.empty_like(o["q"])
    sf = torch.full_like(o["sf"], 0xEE) if "sf" in o else None
    amax = torch.zeros(1, device=dev)
    fp8q.fp8q_residual_norm_quantize_amax(e["residual"], e["residual"], block=d["block"], post_weight=d["post"], gate=d["gate"],
                                          rows_per_gate=per, alpha=0.7, pre_weight=d["pre"], q=q, sf=sf, fmt=fmt, scale=o["scale"], amax=amax)
    assert torch.equal(e["residual"], o["ro"]) and torch.equal(q, o["q"]) and torch.equal(amax, o["amax"])
    assert sf is None or torch.equal(sf, o["sf"])


@pytest.mark.parametrize("rows,H", [(6, 64), (35, 4096), (4, 10000)])
@pytest.mark.parametrize("parts", [dict(block=False), dict(post=False), dict(pre=False), dict(want_q=False), dict(post=False, pre=False)])
def test_forward_parts(dev, rows, H, parts):
    for gate in (None, "f32"):
        if parts.get("block") is False and gate:
            continue
        d = make(rows, H, 2, gate, rows, dev)
        o = forward(d, rows, H, 2, -1.25, 1e-5, dev=dev, **parts)
        check_forward(d, o, rows, H, 2, -1.25, 1e-5, block=parts.get("block", True), post=parts.get("post", True))


def test_forward_h_alone_leaves_the_residual(dev):
    d = make(5, 96, 0, None, 3, dev)
    h, amax = torch.empty(5, 96, dtype=torch.bfloat16, device=dev), torch.zeros(1, device=dev)
    fp8q.fp8q_residual_norm_quantize_amax(d["residual"], None, pre_weight=d["pre"], h=h, amax=amax)
    v = d["residual"].double()
    w = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6) * d["pre"].double()
    near_bf16(h, w, 44 * U * w.abs(), "h")


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
def test_forward_zeros_keep_their_sign(dev, fmt):
    d = make(4, 256, 4, None, 21, dev)
    d["residual"][:, ::3] = -0.0
    d["residual"][:, 1::6] = 0.0
    o = forward(d, 4, 256, 4, 1.0, 1e-6, fmt=fmt, block=False, dev=dev)
    check_forward(d, o, 4, 256, 4, 1.0, 1e-6, fmt, block=False)
    assert (bf16_bits_of(o["h"]) == 0x8000).any()


@pytest.mark.parametrize("fmt", [0, 3])
@pytest.mark.parametrize("H", [64, 4096])
def test_forward_degenerate_rows(dev, H, fmt):
    """Rows of zeros, NaN, infinities and the largest values beside ordinary ones: each keeps to its own row."""
    d = make(12, H, 12, "f32", 5, dev)
    d["block"][1] = 0
    d["residual"][1] = 0
    d["block"][3, 5] = float("nan")
    d["block"][5, 7] = float("inf")
    d["residual"][7, 9] = float("-inf")
    d["residual"][9, 0] = float("nan")
    o = forward(d, 12, H, 12, 1.0, 1e-6, fmt=fmt, dev=dev)
    assert not o["ro"][1].any() and not o["h"][1].any()
    for row in (3, 5, 7, 9):
        assert torch.isnan(o["h"][row]).any()
    ok = torch.tensor([0, 2, 4, 6, 8, 10, 11], device=dev)
    assert torch.isfinite(o["ro"][ok]).all() and torch.isfinite(o["h"][ok]).all()
    assert torch.isnan(o["amax"]).all()
    clean = make(12, H, 12, "f32", 5, dev)
    p = forward(clean, 12, H, 12, 1.0, 1e-6, fmt=fmt, dev=dev)
    assert torch.equal(p["ro"][ok], o["ro"][ok]) and torch.equal(p["h"][ok], o["h"][ok])


def reference_backward(d, s, rows, H, per, alpha):
    """float64 gradients and, for each, the bound that the module's comment derives."""
    z = torch.zeros((rows, H), dtype=torch.float64, device=d["residual"].device)
    dr = s["dro"].double() if s["dro"] is not None else z
    D, dn, n2, E = dr.clone(), z, z, 2 * U * dr.abs()
    out = {}
    strips = 2 + -(-rows // 32)  # additions that a column's term passes through: at most this, and 304 / 32 + 32
    m = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    if s["dh"] is not None:
        r2 = s["rstd_pre"].double()[:, None]
        n2 = s["ro"].double() * r2
        dn = s["dh"].double() * d["pre"].double()
        c2 = m(dn * n2)
        D = dr + r2 * (dn - n2 * c2)
        E = 6 * U * (dr.abs() + r2 * (dn.abs() + (n2 * c2).abs())) + r2 * n2.abs() * 76 * U * m((dn * n2).abs())
        t = s["dh"].double() * n2
        out["d_pre_weight"] = (t.sum(0), (strips + 46) * U * t.abs().sum(0))
    out["d_residual"] = (D, E)
    if s["block"]:
        post = d["post"].double() if s["post"] else torch.ones(H, dtype=torch.float64, device=z.device)
        r1 = s["rstd_post"].double()[:, None] if s["post"] else torch.ones((rows, 1), dtype=torch.float64, device=z.device)
        g = gate_rows(d["gate"], rows, per)
        n1 = d["block"].double() * r1
        e = alpha * g * D
        Ee = (alpha * g * torch.ones_like(D)).abs() * E + 4 * U * e.abs()
        w = alpha * g * post * n1
        eg = e * post
        if s["post"]:
            r2a = s["rstd_pre"].double()[:, None] if s["dh"] is not None else 0.0
            c1 = m(w * D)
            c2a = m(dn * n2).abs()
            big = m((w * dr).abs()) + r2a * m((w * dn).abs()) + r2a * c2a * m((w * n2).abs())
            Ec = 84 * U * (big + r2a * m((dn * n2).abs()) * m((w * n2).abs()))
            db = r1 * (eg - n1 * c1)
            Eb = r1 * (Ee * post.abs() + 4 * U * (eg.abs() + (n1 * c1).abs()) + n1.abs() * Ec) + 2 * U * db.abs()
            t = e * n1
            out["d_post_weight"] = (t.sum(0), (strips + 48) * U * t.abs().sum(0) + (Ee * n1.abs()).sum(0))
        else:
            db, Eb = e, Ee
        out["d_block"] = (db, Eb)
        if d["gate"] is not None:
            t = alpha * D * n1 * post
            at = torch.arange(rows, device=z.device) // per
            zero = torch.zeros(d["gate"].shape, dtype=torch.float64, device=z.device)
            k = (strips + 50) * U
            out["d_gate"] = (zero.clone().index_add_(0, at, t),
                             zero.index_add_(0, at, k * t.abs() + abs(alpha) * E * (n1 * post).abs()))
    return out


def backward(d, s, rows, H, per, alpha, dev):
    bf = lambda: torch.full((rows, H), 7.0, dtype=torch.bfloat16, device=dev)  # noqa: E731
    o = {"d_residual": bf()}
    kw = {}
    if s["dh"] is not None:
        o["d_pre_weight"] = torch.empty(H, device=dev)
    if s["block"]:
        o["d_block"] = bf()
        kw = dict(block=d["block"], gate=d["gate"], rows_per_gate=per, alpha=alpha, d_block=o["d_block"])
        if s["post"]:
            o["d_post_weight"] = torch.empty(H, device=dev)
            kw |= dict(rstd_post=s["rstd_post"], post_weight=d["post"], d_post_weight=o["d_post_weight"])
        if d["gate"] is not None:
            o["d_gate"] = kw["d_gate"] = torch.full_like(d["gate"], 7.0)
    n = fp8q.residual_norm_backward_workspace(rows, H, per if s["block"] and d["gate"] is not None else 0)
    room = torch.full((n + 64,), 0xEE, dtype=torch.uint8, device=dev)
    h = s["dh"] is not None
    fp8q.fp8q_residual_norm_backward(s["dro"], s["dh"], s["ro"] if h else None, s["rstd_pre"] if h else None, d["pre"] if h else None,
                                     o["d_residual"], o.get("d_pre_weight"), workspace=room[:n], **kw)
    assert (room[n:] == 0xEE).all(), "write outside the workspace"
    return o


def check_backward(dev, rows, H, per, gate, alpha=0.7, dh=True, dro=True, block=True, post=True):
    d = make(rows, H, per, gate, rows + H, dev)
    o = forward(d, rows, H, per, alpha, 1e-6, block=block, post=post, want_q=False, dev=dev)
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    f = lambda: torch.randn((rows, H), generator=g, device=dev).bfloat16()  # noqa: E731
    s = {"ro": o["ro"], "rstd_pre": o["rstd_pre"], "rstd_post": o.get("rstd_post"), "dh": f() if dh else None, "dro": f() if dro else None,
         "block": block, "post": post}
    got = backward(d, s, rows, H, per, alpha, dev)
    want = reference_backward(d, s, rows, H, per, alpha)
    assert got.keys() == want.keys()
    for name, (w, bound) in want.items():
        if got[name].dtype == torch.bfloat16:
            near_bf16(got[name], w, bound, name)
        else:
            near_f32(got[name], w, bound, name)
    again = backward(d, s, rows, H, per, alpha, dev)
    for name in got:
        assert torch.equal(again[name], got[name]), f"{name}: the same call gave other bits"


@pytest.mark.parametrize("gate", ["f32", "bf16"])
@pytest.mark.parametrize("rows,H", SHAPES + [(700, 4096), (1500, 512), (3001, 32)])
def test_backward(dev, rows, H, gate):
    per = {16: 1, 48: 2, 256: rows, 512: 7, 528: 1, 80: 11, 1040: 67, 2048: 3, 4096: 100, 32: 1000}.get(H, max(1, rows // 2))
    check_backward(dev, rows, H, per, gate)


@pytest.mark.parametrize("per", [1, 2, 3, 5, 50, 304, 305, 609, 700])
def test_backward_groups_across_strips(dev, per):
    check_backward(dev, 700, 4096, per, "f32")


@pytest.mark.parametrize("parts", [dict(dh=False), dict(dro=False), dict(block=False), dict(post=False), dict(dh=False, post=False)])
@pytest.mark.parametrize("rows,H", [(33, 128), (310, 4096), (9, 9008)])
def test_backward_parts(dev, rows, H, parts):
    check_backward(dev, rows, H, 4, None if parts.get("block") is False else "f32", alpha=-1.5, **parts)
    if parts.get("block") is not False:
        check_backward(dev, rows, H, 4, None, **parts)


PARTS = [dict(), dict(block=False), dict(post=False), dict(pre=False)]


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("rows,H", [(700, 1040), (1900, 2064), (1300, 2560), (900, 4624), (700, 5120), (500, 8208), (350, 10256)])
def test_forward_rows_of_any_number_of_warps(dev, rows, H, parts):
    """Rows that take other numbers of threads than a power of two, several rows a strip, and the call's parts."""
    for fmt in (0, 3):
        for per in (1, 100):
            if parts.get("pre") is False and fmt:
                continue
            d = make(rows, H, per, None if parts.get("block") is False else "bf16", rows + per, dev)
            o = forward(d, rows, H, per, 0.9, 1e-6, fmt=fmt, dev=dev, **parts)
            check_forward(d, o, rows, H, per, 0.9, 1e-6, fmt, block=parts.get("block", True), post=parts.get("post", True))


@pytest.mark.parametrize("parts", [dict(), dict(dh=False), dict(dro=False), dict(block=False), dict(post=False)])
@pytest.mark.parametrize("rows,H", [(1000, 2064), (470, 2560), (300, 5120)])
def test_backward_rows_of_five_warps(dev, rows, H, parts):
    for per in (1, 3, 90):
        check_backward(dev, rows, H, per, None if parts.get("block") is False else "f32", alpha=-0.8, **parts)


def test_backward_against_differences(dev):
    """The formula's own check: central differences of the float64 forward along random directions."""
    rows, H, per, alpha, eps = 6, 64, 2, 0.7, 1e-6
    d = {k: v.double() if v is not None else None for k, v in make(rows, H, per, "f32", 1, dev).items()}
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    f = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float64)  # noqa: E731
    dro, dh = f(rows, H).bfloat16().double(), f(rows, H).bfloat16().double()

    def loss(x):
        y = x["block"] / torch.sqrt(x["block"].square().mean(1, keepdim=True) + eps) * x["post"]
        ro = x["residual"] + alpha * gate_rows(x["gate"], rows, per) * y
        h = ro / torch.sqrt(ro.square().mean(1, keepdim=True) + eps) * x["pre"]
        return (ro * dro).sum() + (h * dh).sum()

    y = d["block"] / torch.sqrt(d["block"].square().mean(1, keepdim=True) + eps) * d["post"]
    ro = d["residual"] + alpha * gate_rows(d["gate"], rows, per) * y
    s = {"ro": ro, "rstd_pre": 1 / torch.sqrt(ro.square().mean(1) + eps), "rstd_post": 1 / torch.sqrt(d["block"].square().mean(1) + eps),
         "dh": dh, "dro": dro, "block": True, "post": True}
    want = reference_backward(d, s, rows, H, per, alpha)
    for name, grad in (("block", "d_block"), ("residual", "d_residual"), ("post", "d_post_weight"), ("pre", "d_pre_weight"), ("gate", "d_gate")):
        v = f(*d[name].shape)
        step = 1e-5
        diff = (loss({**d, name: d[name] + step * v}) - loss({**d, name: d[name] - step * v})) / (2 * step)
        got = (want[grad][0] * v).sum()
        assert abs(float(diff - got)) <= 1e-6 * float((want[grad][0] * v).abs().sum()), name


def test_streams_and_graph(dev):
    rows, H, per = 50, 1040, 7
    d = make(rows, H, per, "f32", 77, dev)
    want = forward(d, rows, H, per, 0.7, 1e-6, fmt=3, dev=dev)
    s = {"ro": want["ro"], "rstd_pre": want["rstd_pre"], "rstd_post": want["rstd_post"], "dh": want["h"], "dro": d["block"], "block": True, "post": True}
    wgrad = backward(d, s, rows, H, per, 0.7, dev)
    torch.cuda.synchronize()
    o = {k: torch.zeros_like(v) for k, v in want.items()}
    o["scale"] = want["scale"]
    gr = {k: torch.zeros_like(v) for k, v in wgrad.items()}
    space = torch.empty(fp8q.residual_norm_backward_workspace(rows, H, per), dtype=torch.uint8, device=dev)

    def both(stream=None):
        fp8q.fp8q_residual_norm_quantize_amax(d["residual"], o["ro"], block=d["block"], post_weight=d["post"], gate=d["gate"], rows_per_gate=per,
                                              alpha=0.7, pre_weight=d["pre"], h=o["h"], q=o["q"], sf=o["sf"], fmt=3, scale=o["scale"],
                                              amax=o["amax"], rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"], stream=stream)
        fp8q.fp8q_residual_norm_backward(d["block"], o["h"], o["ro"], o["rstd_pre"], d["pre"], gr["d_residual"], gr["d_pre_weight"],
                                         block=d["block"], rstd_post=o["rstd_post"], post_weight=d["post"], gate=d["gate"], rows_per_gate=per,
                                         alpha=0.7, d_block=gr["d_block"], d_post_weight=gr["d_post_weight"], d_gate=gr["d_gate"],
                                         workspace=space, stream=stream)

    def same():
        # scales of no row are never written
        return all(torch.equal(o[k], want[k]) for k in want if k != "sf") and all(torch.equal(gr[k], wgrad[k]) for k in wgrad)

    side = torch.cuda.Stream()
    both(side)
    side.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for _ in range(2):
        for t in list(o.values()) + list(gr.values()):
            if t is not o["scale"]:
                t.zero_()
        g.replay()
        assert same()
