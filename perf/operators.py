"""The cases by which the 4-bit and residual-norm operators are measured.

Operators: microscaled 4-bit quantisation (with its transpose) and its inverse, the
product of two 4-bit operands, and the RMS norms after and before a transformer block
fused with its gate, residual scale and quantisation, forward and backward.

``run`` computes a case in elementary torch operations, or, where ``own`` is true, by
the calls that a user makes of ``fp8q``.  ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

BLOCK = {"mx": 32, "nv": 16}

# Hidden 4096, FFN 16384, 4 sequences of 2048 tokens: the transformer MLP that the
# benchmark's workloads are shaped after.


def listed():
    return [
        # fake-quantised activations of one layer, as calibration and 4-bit-aware training see them
        {"name": "roundtrip_nv_8192x4096", "op": "roundtrip", "fmt": "nv", "rows": 8192, "cols": 4096, "both": False},
        # a ragged tensor and its transpose, both directions in one pass, as a backward pass needs them
        {"name": "roundtrip_mx_both_odd", "op": "roundtrip", "fmt": "mx", "rows": 1187, "cols": 2731, "both": True},
        # decode: one token through the MLP's first layer
        {"name": "linear_nv_1_token", "op": "linear", "fmt": "nv", "m": 1, "n": 16384, "k": 4096},
        # serving: a small batch of tokens through the MLP's second layer
        {"name": "linear_mx_24_tokens", "op": "linear", "fmt": "mx", "m": 24, "n": 4096, "k": 16384},
        # the whole batch through the MLP's first layer
        {"name": "linear_nv_ffn", "op": "linear", "fmt": "nv", "m": 8192, "n": 16384, "k": 4096},
        # a ragged prompt from the residual stream: norms, gate, 4-bit codes and the product that reads them
        {"name": "edge_nv_prompt_1555", "op": "edge", "fmt": "nv", "rows": 1555, "hidden": 4096, "n": 11264,
         "per_gate": 1555},
        # a training step of a small odd layer: output and both gradients, every operand quantised in the step
        {"name": "step_mx_odd", "op": "step", "fmt": "mx", "m": 1000, "n": 2072, "k": 1033},
        # a training step of an attention projection over the whole batch
        {"name": "step_nv_8192", "op": "step", "fmt": "nv", "m": 8192, "n": 4096, "k": 4096},
        # one decoded token between two blocks
        {"name": "norm_1_token", "op": "norm", "rows": 1, "hidden": 4096, "per_gate": 1, "gate": "f32", "h": True},
        # the whole batch between two blocks, a gate for each of the four sequences, FP8 codes alone
        {"name": "norm_8192x4096", "op": "norm", "rows": 8192, "hidden": 4096, "per_gate": 2048, "gate": "f32",
         "h": False},
        # gradients of a ragged batch with a gate for each token
        {"name": "norm_grad_odd_row_gate", "op": "norm_grad", "rows": 777, "hidden": 1552, "per_gate": 1, "gate": "bf16"},
        # gradients of the whole batch, a gate for each of the four sequences
        {"name": "norm_grad_8192x4096", "op": "norm_grad", "rows": 8192, "hidden": 4096, "per_gate": 2048, "gate": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["roundtrip", "linear", "linear", "edge", "step", "norm", "norm_grad"])
    fmt = rng.choice(["mx", "nv"])
    if op == "roundtrip":
        while True:
            r, c = _log(rng, 1, 16384), _log(rng, 1, 16384)
            if r * c <= 8192 * 4096:
                return {"op": op, "fmt": fmt, "rows": r, "cols": c, "both": rng.random() < 0.5}
    if op in ("linear", "step"):
        top = 8192 * 16384 * 4096 // (1 if op == "linear" else 4)
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 16, 16384), _log(rng, 16, 16384)
            if m * n * k <= top and max(m * k, n * k, m * n) <= 8192 * 16384:
                return {"op": op, "fmt": fmt, "m": m, "n": n, "k": k}
    while True:
        r, h = _log(rng, 1, 8192), 16 * _log(rng, 1, 1024)
        if r * h <= 8192 * 4096:
            break
    per = rng.choice([1, r, _log(rng, 1, r)])
    if op == "edge":
        while True:
            n = _log(rng, 16, 16384)
            if r * h * n <= 8192 * 16384 * 4096:
                return {"op": op, "fmt": fmt, "rows": r, "hidden": h, "n": n, "per_gate": per}
    case = {"op": op, "rows": r, "hidden": h, "per_gate": per, "gate": rng.choice(["f32", "bf16"])}
    if op == "norm":
        case["h"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# The 4-bit formats in plain torch operations, 32 bits


def _blocks(x, b):
    """[r, c] in float32 -> [r, blocks, b], the last block filled up with zeros."""
    r, c = x.shape
    return torch.nn.functional.pad(x.float(), (0, -c % b)).view(r, -1, b)


def _e2m1(v):
    """Index 0..7 of the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to |v|, ties to the even index."""
    v = v.abs()
    i = (v > 0.25).to(torch.uint8)
    for t, at in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        i += (v >= t) if at else (v > t)
    return i


def _quantize(x, fmt, scale):
    """Codes [r, blocks, b] (sign in bit 3) and block scales [r, blocks] (as bytes) of x."""
    v = _blocks(x, BLOCK[fmt])
    a = v.abs().amax(-1)
    if fmt == "mx":
        e = (torch.frexp(a.clamp(max=3.3895313892515355e38))[1] - 3).clamp(min=-127)
        e = torch.where(a > 0, e, torch.full_like(e, -127))
        u = torch.ldexp(v, -e[..., None])
        sf = (e + 127).to(torch.uint8)
    else:
        s8 = (a / (scale * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = (s8.float() * scale)[..., None]
        u = torch.where(d > 0, v / d, torch.zeros_like(v))
        sf = s8.view(torch.uint8)
    return _e2m1(u) | (torch.signbit(v).to(torch.uint8) << 3), sf


def _values(codes, sf, fmt, scale, c):
    """float32 [r, c]: what codes [r, blocks, b] and block scales stand for."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    v = grid[(codes & 7).int()]
    v = torch.where((codes & 8) != 0, -v, v)
    s = torch.ldexp(torch.ones_like(sf, dtype=torch.float32), sf.int() - 127) if fmt == "mx" else sf.view(torch.float8_e4m3fn).float()
    v = (v * s[..., None]).reshape(codes.shape[0], -1)[:, :c]
    return v if scale is None else v * scale


def _sf_place(r, c, device):
    """Byte offset of the block scale (row, block) in the 128x4-tiled layout, [r, c]."""
    i = torch.arange(r, device=device)[:, None]
    j = torch.arange(c, device=device)[None, :]
    return ((i // 128) * (-(-c // 4)) + j // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4


def _pack(codes, sf, cols):
    """The packed operand that fp8q's 4-bit calls take: codes [r, 16 * ceil(cols / 32)] and tiled block scales."""
    r = codes.shape[0]
    flat = codes.view(r, -1)
    flat = torch.nn.functional.pad(flat, (0, 32 * (-(-cols // 32)) - flat.shape[1]))
    q = flat[:, 0::2] | (flat[:, 1::2] << 4)
    out = torch.zeros(-(-r // 128) * (-(-sf.shape[1] // 4)) * 512, dtype=torch.uint8, device=codes.device)
    out[_sf_place(r, sf.shape[1], codes.device).reshape(-1)] = sf.reshape(-1)
    return q.contiguous(), out


def _unpack(q, sf, cols, fmt):
    """_pack's inverse."""
    r, b = q.shape[0], BLOCK[fmt]
    n = -(-cols // b)
    flat = torch.stack((q & 15, q >> 4), -1).view(r, -1)[:, : n * b]
    return flat.reshape(r, n, b), sf[_sf_place(r, n, q.device)]


# ---------------------------------------------------------------------------
# Inputs


def _activations(shape, g):
    """Activations with a few channels an order of magnitude above the rest."""
    x = torch.randn(shape, generator=g, device="cuda")
    ch = torch.rand(shape[-1], generator=g, device="cuda")
    return (x * torch.where(ch > 0.99, 12.0, 0.5 + ch)).to(torch.bfloat16)


def _scale(x, fmt):
    """The tensor scale of delayed scaling: amax / (6 * 448), which puts the largest block scale at the top of e4m3."""
    return (x.abs().amax().float() / 2688.0).reshape(1) if fmt == "nv" else None


def _norm_inputs(c, g):
    r, h = c["rows"], c["hidden"]
    groups = -(-r // c["per_gate"])
    f = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    gate = 0.5 + 0.25 * f(groups, h)
    return {"block": _activations((r, h), g), "residual": (2.0 * f(r, h)).to(torch.bfloat16),
            "post": 1 + 0.1 * f(h), "pre": 1 + 0.1 * f(h), "gate": gate.to(torch.bfloat16) if c.get("gate") == "bf16" else gate}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c, op = dict(case), case["op"]
    zero = lambda: torch.zeros(1, device="cuda")  # noqa: E731
    if op == "roundtrip":
        x = _activations((c["rows"], c["cols"]), g)
        return {**c, "x": x, "scale": _scale(x, c["fmt"]), "amax": zero()}
    if op in ("linear", "edge"):
        k = c["k"] if op == "linear" else c["hidden"]
        w = (torch.randn((c["n"], k), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
        ws = _scale(w, c["fmt"])
        wq, wsf = _pack(*_quantize(w, c["fmt"], ws), k)
        s = {**c, "wq": wq, "wsf": wsf, "w_scale": ws, "amax": zero()}
        if op == "linear":
            s["x"] = _activations((c["m"], k), g)
            s["scale"] = _scale(s["x"], c["fmt"])
        else:
            s |= _norm_inputs(c, g)
            # delayed scaling: the last step's amax, about the largest of a unit-variance row
            s["scale"] = torch.full((1,), 6.0 / 2688.0, device="cuda") if c["fmt"] == "nv" else None
        return s
    if op == "step":
        x, dy = _activations((c["m"], c["k"]), g), _activations((c["m"], c["n"]), g)
        w = (torch.randn((c["n"], c["k"]), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
        dy = (dy.float() * 1e-3).to(torch.bfloat16)
        return {**c, "x": x, "w": w, "dy": dy, **{n + "_scale": _scale(t, c["fmt"]) for n, t in (("x", x), ("w", w), ("dy", dy))},
                "amax": torch.zeros(3, device="cuda")}
    s = {**c, **_norm_inputs(c, g), "alpha": 0.7, "eps": 1e-6}
    if op == "norm":
        return {**s, "scale": torch.full((1,), 5.0 / 448.0, device="cuda"), "amax": zero()}
    # what the forward pass leaves behind for the backward one
    b, gate = s["block"].float(), s["gate"].float()
    s["rstd_post"] = torch.rsqrt((b * b).mean(-1) + s["eps"])
    rows = torch.arange(c["rows"], device="cuda") // c["per_gate"]
    new = s["residual"].float() + s["alpha"] * gate[rows] * (b * s["rstd_post"][:, None] * s["post"])
    s["residual_out"] = new.to(torch.bfloat16)
    new = s["residual_out"].float()
    s["rstd_pre"] = torch.rsqrt((new * new).mean(-1) + s["eps"])
    s["d_out"] = _activations((c["rows"], c["hidden"]), g)
    s["d_h"] = _activations((c["rows"], c["hidden"]), g)
    return s


# ---------------------------------------------------------------------------
# The plain forms


def _norm_plain(s, alpha, eps):
    rows = torch.arange(s["rows"], device="cuda") // s["per_gate"]
    b = s["block"].float()
    y = b * torch.rsqrt((b * b).mean(-1, keepdim=True) + eps) * s["post"]
    new = (s["residual"].float() + alpha * s["gate"].float()[rows] * y).to(torch.bfloat16)
    v = new.float()
    h = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps) * s["pre"]).to(torch.bfloat16)
    return new, h


def _groups(x, per):
    """Sum of [rows, h] over each run of `per` rows."""
    r, h = x.shape
    return torch.nn.functional.pad(x, (0, 0, 0, -r % per)).view(-1, per, h).sum(1)


def _plain(s):
    op, fmt = s["op"], s.get("fmt")
    if op == "roundtrip":
        x, sc = s["x"], s["scale"]
        y = _values(*_quantize(x, fmt, sc), fmt, sc, x.shape[1]).to(torch.bfloat16)
        amax = x.abs().amax().float().reshape(1)
        if not s["both"]:
            return {"y": y, "amax": amax}
        t = x.t()
        return {"y": y, "yt": _values(*_quantize(t, fmt, sc), fmt, sc, t.shape[1]).to(torch.bfloat16), "amax": amax}
    if op in ("linear", "edge"):
        out = {}
        if op == "edge":
            out["residual"], x = _norm_plain(s, 1.0, 1e-6)
        else:
            x = s["x"]
        k = x.shape[1]
        a = _values(*_quantize(x, fmt, s["scale"]), fmt, s["scale"], k)
        w = _values(*_unpack(s["wq"], s["wsf"], k, fmt), fmt, s["w_scale"], k)
        return {**out, "y": (a @ w.t()).to(torch.bfloat16), "amax": x.abs().amax().float().reshape(1)}
    if op == "step":
        v = {}
        for n in ("x", "w", "dy"):
            t, sc = s[n], s[n + "_scale"]
            v[n] = _values(*_quantize(t, fmt, sc), fmt, sc, t.shape[1])
            v[n + "t"] = _values(*_quantize(t.t(), fmt, sc), fmt, sc, t.shape[0])
        return {"y": (v["x"] @ v["w"].t()).to(torch.bfloat16), "dx": (v["dy"] @ v["wt"].t()).to(torch.bfloat16),
                "dw": (v["dyt"] @ v["xt"].t()).to(torch.bfloat16),
                "amax": torch.stack([s[n].abs().amax().float() for n in ("x", "w", "dy")])}
    if op == "norm":
        new, h = _norm_plain(s, s["alpha"], s["eps"])
        q = (h.float() / s["scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        out = {"residual": new, "q": q, "amax": h.abs().amax().float().reshape(1)}
        return {**out, "h": h} if s["h"] else out
    rows = torch.arange(s["rows"], device="cuda") // s["per_gate"]
    n2 = s["residual_out"].float() * s["rstd_pre"][:, None]
    dh = s["d_h"].float()
    dn = dh * s["pre"]
    D = s["d_out"].float() + s["rstd_pre"][:, None] * (dn - n2 * (dn * n2).mean(-1, keepdim=True))
    n1 = s["block"].float() * s["rstd_post"][:, None]
    e = s["alpha"] * s["gate"].float()[rows] * D
    eg = e * s["post"]
    db = s["rstd_post"][:, None] * (eg - n1 * (eg * n1).mean(-1, keepdim=True))
    return {"d_residual": D.to(torch.bfloat16), "d_block": db.to(torch.bfloat16), "d_pre": (dh * n2).sum(0),
            "d_post": (e * n1).sum(0), "d_gate": _groups(s["alpha"] * D * n1 * s["post"], s["per_gate"]).to(s["gate"].dtype)}


# ---------------------------------------------------------------------------
# The framework's calls


def _own(s):
    from quantize_amax_scaling_gb300 import fp8q
    op = s["op"]
    fmt = {"mx": fp8q.MXFP4, "nv": fp8q.NVFP4, None: None}[s.get("fmt")]
    bf = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    if op == "roundtrip":
        x = s["x"]
        r, c = x.shape
        q, sf = fp8q.fp4_empty(r, c, fmt)
        qt, sft = fp8q.fp4_empty(c, r, fmt) if s["both"] else (None, None)
        fp8q.fp8q_fp4_quantize_amax(x, q, sf, fmt, s["scale"], s["amax"], qt=qt, sft=sft)
        out = {"y": bf(r, c), "amax": s["amax"]}
        fp8q.fp8q_fp4_dequantize(q, sf, out["y"], fmt, s["scale"])
        if s["both"]:
            out["yt"] = bf(c, r)
            fp8q.fp8q_fp4_dequantize(qt, sft, out["yt"], fmt, s["scale"])
        return out
    if op in ("linear", "edge"):
        m, k = (s["m"], s["k"]) if op == "linear" else (s["rows"], s["hidden"])
        q, sf = fp8q.fp4_empty(m, k, fmt)
        out = {"y": bf(m, s["n"]), "amax": s["amax"]}
        if op == "linear":
            fp8q.fp8q_fp4_quantize_amax(s["x"], q, sf, fmt, s["scale"], s["amax"])
        else:
            out["residual"] = bf(m, k)
            fp8q.fp8q_residual_norm_quantize_amax(
                s["residual"], out["residual"], block=s["block"], post_weight=s["post"], gate=s["gate"],
                rows_per_gate=s["per_gate"], alpha=1.0, pre_weight=s["pre"], q=q, sf=sf, fmt=fmt, scale=s["scale"],
                amax=s["amax"], eps=1e-6)
        fp8q.fp8q_fp4_matmul(q, sf, s["wq"], s["wsf"], out["y"], k, fmt, s["scale"], s["w_scale"])
        return out
    if op == "step":
        m, n, k = s["m"], s["n"], s["k"]
        shapes = {"x": (m, k), "w": (n, k), "dy": (m, n)}
        p = {}
        for i, (name, (r, c)) in enumerate(shapes.items()):
            p[name], p[name + "t"] = fp8q.fp4_empty(r, c, fmt), fp8q.fp4_empty(c, r, fmt)
            fp8q.fp8q_fp4_quantize_amax(s[name], *p[name], fmt, s[name + "_scale"], s["amax"][i : i + 1],
                                        qt=p[name + "t"][0], sft=p[name + "t"][1])
        out = {"y": bf(m, n), "dx": bf(m, k), "dw": bf(n, k), "amax": s["amax"]}
        fp8q.fp8q_fp4_matmul(*p["x"], *p["w"], out["y"], k, fmt, s["x_scale"], s["w_scale"])
        fp8q.fp8q_fp4_matmul(*p["dy"], *p["wt"], out["dx"], n, fmt, s["dy_scale"], s["w_scale"])
        fp8q.fp8q_fp4_matmul(*p["dyt"], *p["xt"], out["dw"], m, fmt, s["dy_scale"], s["x_scale"])
        return out
    r, h = s["rows"], s["hidden"]
    if op == "norm":
        out = {"residual": bf(r, h), "q": torch.empty((r, h), dtype=torch.float8_e4m3fn, device="cuda"), "amax": s["amax"]}
        if s["h"]:
            out["h"] = bf(r, h)
        fp8q.fp8q_residual_norm_quantize_amax(
            s["residual"], out["residual"], block=s["block"], post_weight=s["post"], gate=s["gate"],
            rows_per_gate=s["per_gate"], alpha=s["alpha"], pre_weight=s["pre"], h=out.get("h"), q=out["q"],
            fmt=fp8q.E4M3FN, scale=s["scale"], amax=s["amax"], eps=s["eps"])
        return out
    out = {"d_residual": bf(r, h), "d_block": bf(r, h), "d_pre": torch.empty(h, device="cuda"),
           "d_post": torch.empty(h, device="cuda"), "d_gate": torch.empty_like(s["gate"])}
    space = torch.empty(fp8q.residual_norm_backward_workspace(r, h, s["per_gate"]), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_residual_norm_backward(
        s["d_out"], s["d_h"], s["residual_out"], s["rstd_pre"], s["pre"], out["d_residual"], out["d_pre"],
        block=s["block"], rstd_post=s["rstd_post"], post_weight=s["post"], gate=s["gate"], rows_per_gate=s["per_gate"],
        alpha=s["alpha"], d_block=out["d_block"], d_post_weight=out["d_post"], d_gate=out["d_gate"], workspace=space)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    c, op = case, case["op"]
    per = {"mx": 0.5 + 1 / 32, "nv": 0.5 + 1 / 16, None: 0}[c.get("fmt")]
    if op == "roundtrip":
        n = c["rows"] * c["cols"]
        k = 2 if c["both"] else 1
        return {"bytes": n * 2 + k * n * (per + 2), "flops": 4 * k * n}
    if op == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * m * k + per * n * k + 2 * m * n, "flops": 2 * m * n * k}
    if op == "edge":
        m, n, k = c["rows"], c["n"], c["hidden"]
        return {"bytes": 6 * m * k + 4 * k * (2 + -(-m // c["per_gate"])) + per * n * k + 2 * m * n, "flops": 2 * m * n * k + 12 * m * k}
    if op == "step":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * (m * k + n * k + m * n) * 2, "flops": 6 * m * n * k}
    n, h = c["rows"] * c["hidden"], c["hidden"]
    gate = -(-c["rows"] // c["per_gate"]) * h * (2 if c["gate"] == "bf16" else 4)
    if op == "norm":
        return {"bytes": n * (7 + (2 if c["h"] else 0)) + gate + 8 * h, "flops": 14 * n}
    return {"bytes": 12 * n + 2 * gate + 16 * h + 8 * c["rows"], "flops": 30 * n}


# ---------------------------------------------------------------------------
# The definitions in 64 bits

_TOP = 448.0


def _e4m3_64(v):
    """Nearest e4m3 value of v >= 0 in float64, ties to even, held at 448."""
    step = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(max=_TOP)


def _fp4_64(x, fmt, scale):
    """The values that the 4-bit codes of x stand for, float64 [r, c].  The quotients that the definition
    rounds to binary32 are rounded from 64 bits: a quotient of two binary32 numbers is not changed by that."""
    r, c = x.shape
    b = BLOCK[fmt]
    pad = torch.zeros((r, -c % b), dtype=torch.float64, device=x.device)
    v = torch.cat((x.double(), pad), 1).reshape(r, -1, b)
    a = v.abs().amax(2, keepdim=True)
    if fmt == "mx":
        # the floor of the logarithm, put right where log2 rounded across a power of two
        e = torch.floor(torch.log2(a.clamp(min=2.0 ** -140)))
        e = e - (torch.exp2(e) > a).double() + (torch.exp2(e + 1) <= a).double()
        d = torch.exp2((e - 2).clamp(min=-127))
        u, s = v / d, 1.0
    else:
        s = scale.double()
        s8 = _e4m3_64((a / (6 * s).float().double()).float().double())
        d = s8
        by = (s8 * s).float().double()
        u = (v / by.clamp(min=1e-300)).float().double() * (by > 0)
    m = u.abs().clamp(max=6.0)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    m = (torch.round(m / step) * step).clamp(max=6.0)
    return (torch.copysign(m, v) * d).reshape(r, -1)[:, :c] * s


def _norm_64(s, alpha, eps):
    at = torch.div(torch.arange(s["rows"], device="cuda"), s["per_gate"], rounding_mode="floor")
    b = s["block"].double()
    y = b / torch.sqrt(b.square().mean(1, keepdim=True) + eps) * s["post"].double()
    new = s["residual"].double() + alpha * s["gate"].double()[at] * y
    v = new.to(torch.bfloat16).double()
    return new, v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * s["pre"].double()


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = s["op"], s.get("fmt")
    top = lambda t: t.double().abs().max().reshape(1)  # noqa: E731
    if op == "roundtrip":
        out = {"y": _fp4_64(s["x"], fmt, s["scale"]), "amax": top(s["x"])}
        return {**out, "yt": _fp4_64(s["x"].t().contiguous(), fmt, s["scale"])} if s["both"] else out
    if op in ("linear", "edge"):
        out = {}
        if op == "edge":
            out["residual"], x = _norm_64(s, 1.0, 1e-6)
            out["amax"] = top(x.to(torch.bfloat16))
            x = x.to(torch.bfloat16)
        else:
            x = s["x"]
            out["amax"] = top(x)
        k = x.shape[1]
        nib = torch.cat(((s["wq"] & 15)[..., None], (s["wq"] >> 4)[..., None]), 2).flatten(1)[:, :k].long()
        val = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")[nib]
        nb = -(-k // BLOCK[fmt])
        tiles = s["wsf"].view(-(-s["n"] // 128), -(-nb // 4), 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-(-s["n"] // 128) * 128, -1)
        tiles = tiles[: s["n"], :nb].contiguous()
        sf = torch.exp2(tiles.double() - 127) if fmt == "mx" else tiles.view(torch.float8_e4m3fn).double()
        w = val * sf.repeat_interleave(BLOCK[fmt], 1)[:, :k] * (1.0 if fmt == "mx" else s["w_scale"].double())
        out["y"] = _fp4_64(x, fmt, s["scale"]) @ w.t()
        return out
    if op == "step":
        f = lambda n, t: _fp4_64(s[n].t().contiguous() if t else s[n], fmt, s[n + "_scale"])  # noqa: E731
        return {"y": f("x", 0) @ f("w", 0).t(), "dx": f("dy", 0) @ f("w", 1).t(), "dw": f("dy", 1) @ f("x", 1).t(),
                "amax": torch.cat([top(s[n]) for n in ("x", "w", "dy")])}
    if op == "norm":
        new, h = _norm_64(s, s["alpha"], s["eps"])
        out = {"residual": new, "q": (h / s["scale"].double()).clamp(-_TOP, _TOP), "amax": top(h.to(torch.bfloat16))}
        return {**out, "h": h} if s["h"] else out
    at = torch.div(torch.arange(s["rows"], device="cuda"), s["per_gate"], rounding_mode="floor")
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    r2, r1 = d["rstd_pre"].unsqueeze(1), d["rstd_post"].unsqueeze(1)
    h, gate = s["hidden"], d["gate"][at]
    n2, n1 = d["residual_out"] * r2, d["block"] * r1
    dn = d["d_h"] * d["pre"]
    D = d["d_out"] + r2 * dn - r2 * n2 * ((dn * n2).sum(1, keepdim=True) / h)
    dy = s["alpha"] * gate * D
    dn1 = dy * d["post"]
    db = r1 * dn1 - r1 * n1 * ((dn1 * n1).sum(1, keepdim=True) / h)
    dg = torch.zeros_like(d["gate"]).index_add_(0, at, s["alpha"] * D * n1 * d["post"])
    return {"d_residual": D, "d_block": db, "d_pre": (d["d_h"] * n2).sum(0), "d_post": (dy * n1).sum(0), "d_gate": dg}
