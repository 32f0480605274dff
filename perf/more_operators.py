"""The cases by which the 8-bit products, the products grouped by expert and the 8-bit checkpoints are measured.

Operators: the product of two FP8 operands with bias, GELU, residual, FP8 codes and a checkpoint in its epilogue, in
every orientation of its operands; the same over rows sorted by expert, with the experts' weight gradients; the
checkpoint of an activation in 8 bits (blocks of 32 under a power of two) and the GELU's backward pass from it.

``run`` computes a case in elementary torch operations, or, where ``own`` is true, by the calls that a user makes of
``fp8q``.  ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4: 448.0, E5: 57344.0}

# Hidden 4096, FFN 16384, 4 sequences of 2048 tokens: the transformer MLP that the benchmark's workloads are shaped
# after.  The experts' sizes are generic.


def listed():
    return [
        # decode: one token through the MLP's first layer, straight into the codes that the second one reads
        {"name": "up_1_token", "op": "linear", "m": 1, "n": 16384, "k": 4096, "bias": "f32", "gelu": True,
         "residual": False, "out": "q", "ckpt": False},
        # serving: a small batch of tokens through the second layer and into the residual stream
        {"name": "down_24_tokens", "op": "linear", "m": 24, "n": 4096, "k": 16384, "bias": "bf16", "gelu": False,
         "residual": True, "out": "bf16", "ckpt": False},
        # training: the whole batch through the first layer, the GELU's input kept in 8 bits (and read back)
        {"name": "up_8192_checkpoint", "op": "linear", "m": 8192, "n": 16384, "k": 4096, "bias": "f32", "gelu": True,
         "residual": False, "out": "q", "ckpt": True},
        # both gradient products of a ragged batch through a small layer, the weight's added to what other
        # micro-batches left
        {"name": "grads_ragged", "op": "grads", "m": 1003, "n": 2064, "k": 1040},
        # both gradient products of an attention projection over the whole batch
        {"name": "grads_8192", "op": "grads", "m": 8192, "n": 4096, "k": 4096},
        # decode: 24 tokens, two experts of sixteen each
        {"name": "experts_48_rows", "op": "experts", "rows": 48, "experts": 16, "hidden": 2048, "ffn": 4096},
        # prefill: 8192 tokens, two experts of eight each
        {"name": "experts_16384_rows", "op": "experts", "rows": 16384, "experts": 8, "hidden": 4096, "ffn": 4096},
        # a training step's gradients of a small layer of experts, some without rows
        {"name": "experts_grads", "op": "experts_grads", "rows": 3001, "experts": 12, "n": 2064, "k": 1040},
        # an activation of the whole batch kept in 8 bits and read back
        {"name": "checkpoint_8192x4096", "op": "checkpoint", "rows": 8192, "cols": 4096},
        # a ragged one
        {"name": "checkpoint_odd", "op": "checkpoint", "rows": 1187, "cols": 2731},
        # back through the GELU of the whole batch, from the checkpoint: gradient codes and the bias's gradient
        {"name": "gelu_back_8192x16384", "op": "gelu_back", "rows": 8192, "cols": 16384, "fmt": "e5"},
        # back through that of a small ragged batch
        {"name": "gelu_back_ragged", "op": "gelu_back", "rows": 777, "cols": 1552, "fmt": "e4"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grads", "experts", "experts_grads", "checkpoint", "gelu_back"])
    if op == "linear":
        while True:
            m, n, k = _log(rng, 1, 8192), 16 * _log(rng, 1, 1024), 16 * _log(rng, 1, 1024)
            if m * n * k <= 8192 * 16384 * 4096 and max(m * k, n * k, m * n) <= 8192 * 16384:
                break
        gelu = rng.random() < 0.5
        return {"op": op, "m": m, "n": n, "k": k, "bias": rng.choice(["none", "f32", "bf16"]), "gelu": gelu,
                "residual": rng.random() < 0.5, "out": rng.choice(["q", "bf16", "both"]), "ckpt": gelu and rng.random() < 0.5}
    if op == "grads":
        while True:
            m, n, k = _log(rng, 1, 8192), 16 * _log(rng, 1, 1024), 16 * _log(rng, 1, 1024)
            if m * n * k <= 8192 * 4096 * 8192 and max(m * k, n * k, m * n) <= 8192 * 16384:
                return {"op": op, "m": m, "n": n, "k": k}
    if op in ("experts", "experts_grads"):
        while True:
            rows, e = _log(rng, 1, 16384), _log(rng, 1, 64)
            n, k = 16 * _log(rng, 1, 512), 16 * _log(rng, 1, 512)
            # the plain form gathers each expert's rows into as many as the fullest has
            if rows * n * k <= 16384 * 4096 * 4096 and e * n * k <= 16 * 4096 * 4096 and e * rows * max(n, k) <= 64 * 16384 * 512:
                break
        if op == "experts":
            return {"op": op, "rows": rows, "experts": e, "hidden": k, "ffn": n}
        return {"op": op, "rows": rows, "experts": e, "n": n, "k": k}
    while True:
        r, c = _log(rng, 1, 16384), _log(rng, 1, 16384)
        if r * c <= 8192 * 16384:
            return {"op": op, "rows": r, "cols": c, **({"fmt": rng.choice(["e4", "e5"])} if op == "gelu_back" else {})}


# ---------------------------------------------------------------------------
# Inputs


def _activations(shape, g):
    """Activations with a few channels an order of magnitude above the rest."""
    x = torch.randn(shape, generator=g, device="cuda")
    ch = torch.rand(shape[-1], generator=g, device="cuda")
    return x * torch.where(ch > 0.99, 8.0, 0.5 + ch)


def _codes(x, dt):
    """FP8 codes of x and the scale that puts its largest at the top of the format, as delayed scaling does."""
    s = (x.abs().amax() / TOP[dt]).clamp(min=1e-30).reshape(1)
    return (x / s).to(dt), s


def _offsets(rows, e, g):
    """[e + 1] int32: unlike shares, some of them nothing where there are more than a few experts."""
    share = torch.rand(e, generator=g, device="cuda") ** 2
    if e > 3:
        share[torch.randint(e, (1 + e // 8,), generator=g, device="cuda")] = 0.0
    at = torch.cumsum(share, 0) / share.sum().clamp(min=1e-30)
    off = torch.cat((torch.zeros(1, device="cuda"), (at * rows).round().clamp(0, rows)))
    off[-1] = rows
    return off.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c, op = dict(case), case["op"]
    f = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    zero = lambda: torch.zeros(1, device="cuda")  # noqa: E731
    if op == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        a, sa = _codes(_activations((m, k), g), E4)
        b, sb = _codes(f(n, k) / math.sqrt(k), E4)
        s = {**c, "a": a, "sa": sa, "b": b, "sb": sb, "amax": zero(), "q_scale": torch.full((1,), 8.0 / 448, device="cuda")}
        s["bias_t"] = None if c["bias"] == "none" else (0.2 * f(n)).to(torch.bfloat16 if c["bias"] == "bf16" else torch.float32)
        s["res"] = (2.0 * f(m, n)).to(torch.bfloat16) if c["residual"] else None
        return s
    if op == "grads":
        m, n, k = c["m"], c["n"], c["k"]
        x, sx = _codes(_activations((m, k), g), E4)
        w, sw = _codes(f(n, k) / math.sqrt(k), E4)
        dy, sdy = _codes(1e-3 * _activations((m, n), g), E5)
        return {**c, "x": x, "sx": sx, "w": w, "sw": sw, "dy": dy, "sdy": sdy, "dw": 1e-2 * f(n, k)}
    if op == "experts":
        r, e, h, n = c["rows"], c["experts"], c["hidden"], c["ffn"]
        off = _offsets(r, e, g)
        x, sx = _codes(_activations((r, h), g), E4)
        w1, s1 = _codes(f(e, n, h) / math.sqrt(h), E4)
        w2, s2 = _codes(f(e, h, n) / math.sqrt(n), E4)
        return {**c, "off": off, "most": int((off[1:] - off[:-1]).max()), "x": x, "sx": sx, "w1": w1, "s1": s1, "w2": w2,
                "s2": s2, "b1": 0.2 * f(e, n), "amax": zero(), "q_scale": torch.full((1,), 8.0 / 448, device="cuda")}
    if op == "experts_grads":
        r, e, n, k = c["rows"], c["experts"], c["n"], c["k"]
        off = _offsets(r, e, g)
        x, sx = _codes(_activations((r, k), g), E4)
        w, sw = _codes(f(e, n, k) / math.sqrt(k), E4)
        dy, sdy = _codes(1e-3 * _activations((r, n), g), E5)
        return {**c, "off": off, "most": int((off[1:] - off[:-1]).max()), "x": x, "sx": sx, "w": w, "sw": sw, "dy": dy, "sdy": sdy}
    x = _activations((c["rows"], c["cols"]), g).to(torch.bfloat16)
    if op == "checkpoint":
        return {**c, "x": x}
    q, sf = _ckpt(x)
    dt = E4 if c["fmt"] == "e4" else E5
    dy = (1e-3 * _activations((c["rows"], c["cols"]), g)).to(torch.bfloat16)
    # delayed scaling: the last step's amax, about this one's
    return {**c, "h": q, "h_sf": sf, "dy": dy, "scale": (dy.float().abs().amax() / TOP[dt]).reshape(1), "amax": zero()}


# ---------------------------------------------------------------------------
# The plain forms


def _gelu(x):
    """The tanh form."""
    return x / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _gelu_slope(x):
    x = x.clamp(-10.0, 10.0)  # beyond, 0 and 1 to 35 places
    c = 2.0 * math.sqrt(2.0 / math.pi)
    t = torch.exp(-c * (x + 0.044715 * x * x * x))
    s = 1.0 / (1.0 + t)
    return s + x * s * (t * s) * (c * (1.0 + 3 * 0.044715 * x * x))


def _fp8(y, scale, dt):
    """Codes of a bf16 tensor."""
    return (y.float() / scale).clamp(-TOP[dt], TOP[dt]).to(dt)


def _ckpt(x):
    """e4m3 codes [rows, cols] of a bf16 matrix, and its block scales [rows, blocks]: e + 127 of the least 2^e that
    holds the block's largest within 448."""
    r, c = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -c % 32)).view(r, -1, 32)
    a = v.abs().amax(-1)
    m, e = torch.frexp(a)
    e = torch.where(a > 0, (e - 9 + (m > 0.875)).clamp(min=-127), torch.full_like(e, -127))
    q = torch.ldexp(v, -e[..., None]).to(E4)
    return q.view(r, -1)[:, :c].contiguous(), (e + 127).to(torch.uint8)


def _ckpt_value(q, sf):
    """float32 [rows, cols]."""
    r, c = q.shape
    s = torch.ldexp(torch.ones_like(sf, dtype=torch.float32), sf.int() - 127)
    return q.float() * s.repeat_interleave(32, 1)[:, :c]


def _linear_plain(s):
    z = (s["a"].float() @ s["b"].float().t()) * (s["sa"] * s["sb"])
    if s["bias_t"] is not None:
        z = z + s["bias_t"].float()
    y = _gelu(z) if s["gelu"] else z
    if s["res"] is not None:
        y = y + s["res"].float()
    y = y.to(torch.bfloat16)
    out = {}
    if s["out"] != "bf16":
        out["q"] = _fp8(y, s["q_scale"], E4)
        out["amax"] = y.abs().amax().float().reshape(1)
    if s["out"] != "q":
        out["y"] = y
    if s["ckpt"]:
        out["h"] = _ckpt_value(*_ckpt(z.to(torch.bfloat16))).to(torch.bfloat16)
    return out


def _gathered(x, off, most):
    """[experts, most, cols] float32 of rows sorted by expert, zeros where an expert has fewer."""
    at = off[:-1, None].long() + torch.arange(most, device=x.device)
    there = at < off[1:, None]
    return torch.where(there[..., None], x.float()[at.clamp(max=x.shape[0] - 1)], torch.zeros((), device=x.device))


def _back_in_rows(y, off, rows):
    """_gathered's inverse."""
    r = torch.arange(rows, device=y.device)
    e = torch.bucketize(r, off[1:].long(), right=True)
    return y[e, r - off[e].long()]


def _plain(s):
    op = s["op"]
    if op == "linear":
        return _linear_plain(s)
    if op == "grads":
        x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
        return {"dx": ((dy @ w) * (s["sdy"] * s["sw"])).to(torch.bfloat16), "dw": (dy.t() @ x) * (s["sdy"] * s["sx"]) + s["dw"]}
    if op == "experts":
        off, most = s["off"], s["most"]
        z = torch.bmm(_gathered(s["x"], off, most), s["w1"].float().transpose(1, 2)) * (s["sx"] * s["s1"])
        a = _back_in_rows(_gelu(z + s["b1"][:, None]), off, s["rows"]).to(torch.bfloat16)
        q = _fp8(a, s["q_scale"], E4)
        y = torch.bmm(_gathered(q, off, most), s["w2"].float().transpose(1, 2)) * (s["q_scale"] * s["s2"])
        return {"q": q, "amax": a.abs().amax().float().reshape(1), "y": _back_in_rows(y, off, s["rows"]).to(torch.bfloat16)}
    if op == "experts_grads":
        dy, x = _gathered(s["dy"], s["off"], s["most"]), _gathered(s["x"], s["off"], s["most"])
        dx = torch.bmm(dy, s["w"].float()) * (s["sdy"] * s["sw"])
        return {"dx": _back_in_rows(dx, s["off"], s["rows"]).to(torch.bfloat16),
                "dw": torch.bmm(dy.transpose(1, 2), x) * (s["sdy"] * s["sx"])}
    if op == "checkpoint":
        return {"y": _ckpt_value(*_ckpt(s["x"])).to(torch.bfloat16)}
    d = s["dy"].float() * _gelu_slope(_ckpt_value(s["h"], s["h_sf"]))
    y = d.to(torch.bfloat16)
    return {"q": _fp8(y, s["scale"], E4 if s["fmt"] == "e4" else E5), "amax": y.abs().amax().float().reshape(1), "d_bias": d.sum(0)}


# ---------------------------------------------------------------------------
# The framework's calls


def _own(s):
    from quantize_amax_scaling_gb300 import fp8q
    op = s["op"]
    bf = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    if op == "linear":
        m, n = s["m"], s["n"]
        out = {}
        if s["out"] != "bf16":
            out |= {"q": torch.empty((m, n), dtype=E4, device="cuda"), "amax": s["amax"]}
        if s["out"] != "q":
            out["y"] = bf(m, n)
        h, h_sf = fp8q.checkpoint_empty(m, n) if s["ckpt"] else (None, None)
        fp8q.fp8q_matmul(s["a"], s["b"], out.get("y"), fp8q.E4M3FN, fp8q.E4M3FN, s["sa"], s["sb"], bias=s["bias_t"],
                         act=fp8q.ACT_GELU if s["gelu"] else fp8q.ACT_NONE, residual=s["res"], q=out.get("q"), q_fmt=fp8q.E4M3FN,
                         q_scale=s["q_scale"] if "q" in out else None, amax=out.get("amax"), h=h, h_sf=h_sf)
        if s["ckpt"]:
            out["h"] = bf(m, n)
            fp8q.fp8q_checkpoint_dequantize(h, h_sf, out["h"])
        return out
    if op == "grads":
        out = {"dx": bf(s["m"], s["k"]), "dw": torch.empty((s["n"], s["k"]), device="cuda")}
        fp8q.fp8q_matmul(s["dy"], s["w"], out["dx"], fp8q.E5M2, fp8q.E4M3FN, s["sdy"], s["sw"], b_trans=True)
        fp8q.fp8q_matmul(s["dy"], s["x"], out["dw"], fp8q.E5M2, fp8q.E4M3FN, s["sdy"], s["sx"], a_trans=True, b_trans=True,
                         residual=s["dw"])
        return out
    if op == "experts":
        out = {"q": torch.empty((s["rows"], s["ffn"]), dtype=E4, device="cuda"), "amax": s["amax"], "y": bf(s["rows"], s["hidden"])}
        fp8q.fp8q_grouped_matmul(s["x"], s["w1"], s["off"], None, fp8q.E4M3FN, fp8q.E4M3FN, s["sx"], s["s1"], bias=s["b1"],
                                 act=fp8q.ACT_GELU, q=out["q"], q_fmt=fp8q.E4M3FN, q_scale=s["q_scale"], amax=s["amax"])
        fp8q.fp8q_grouped_matmul(out["q"], s["w2"], s["off"], out["y"], fp8q.E4M3FN, fp8q.E4M3FN, s["q_scale"], s["s2"])
        return out
    if op == "experts_grads":
        out = {"dx": bf(s["rows"], s["k"]), "dw": torch.empty((s["experts"], s["n"], s["k"]), device="cuda")}
        fp8q.fp8q_grouped_matmul(s["dy"], s["w"], s["off"], out["dx"], fp8q.E5M2, fp8q.E4M3FN, s["sdy"], s["sw"], b_trans=True)
        fp8q.fp8q_grouped_weight_gradient(s["dy"], s["x"], s["off"], out["dw"], fp8q.E5M2, fp8q.E4M3FN, s["sdy"], s["sx"])
        return out
    r, c = s["rows"], s["cols"]
    if op == "checkpoint":
        h, h_sf = fp8q.checkpoint_empty(r, c)
        out = {"y": bf(r, c)}
        fp8q.fp8q_checkpoint_quantize(s["x"], h, h_sf)
        fp8q.fp8q_checkpoint_dequantize(h, h_sf, out["y"])
        return out
    e4 = s["fmt"] == "e4"
    out = {"q": torch.empty((r, c), dtype=E4 if e4 else E5, device="cuda"), "amax": s["amax"], "d_bias": torch.empty(c, device="cuda")}
    space = torch.empty(fp8q.gelu_backward_workspace(r, c), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_gelu_backward_quantize_amax(s["dy"], s["h"], s["h_sf"], out["q"], fp8q.E4M3FN if e4 else fp8q.E5M2, s["scale"], s["amax"],
                                          d_bias=out["d_bias"], workspace=space)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    c, op = case, case["op"]
    if op == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        per = {"q": 1, "bf16": 2, "both": 3}[c["out"]] + (2 if c["residual"] else 0) + (2 if c["ckpt"] else 0)
        return {"bytes": m * k + n * k + m * n * per + {"none": 0, "f32": 4, "bf16": 2}[c["bias"]] * n, "flops": 2 * m * n * k}
    if op == "grads":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k + n * k + m * n + 2 * m * k + 8 * n * k, "flops": 4 * m * n * k}
    if op == "experts":
        r, e, h, n = c["rows"], min(c["rows"], c["experts"]), c["hidden"], c["ffn"]
        return {"bytes": r * h * 3 + r * n + e * (2 * h * n + 4 * n), "flops": 4 * r * h * n}
    if op == "experts_grads":
        r, e, n, k = c["rows"], c["experts"], c["n"], c["k"]
        return {"bytes": r * (n + k + 2 * k) + min(r, e) * n * k + 4 * e * n * k, "flops": 4 * r * n * k}
    n = c["rows"] * c["cols"]
    if op == "checkpoint":
        return {"bytes": 4 * n, "flops": 3 * n}
    return {"bytes": 4 * n + n / 32 + 4 * c["cols"], "flops": 25 * n}


# ---------------------------------------------------------------------------
# The definitions in 64 bits


def _gelu_64(x):
    u = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return 0.5 * x * (1 + torch.tanh(u))


def _gelu_slope_64(x):
    x = x.clamp(-60, 60)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def _fp8_64(v, dt):
    """Nearest FP8 value of v in float64, ties to even, held at the format's largest."""
    least, bits = (2.0 ** -6, 3) if dt is E4 else (2.0 ** -14, 2)
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=least))) - bits)
    return torch.copysign((torch.round(a / step) * step).clamp(max=TOP[dt]), v)


def _quotient_64(y, scale, dt):
    """What the codes of a bf16 tensor stand for, but for the scale: the quotient is one of binary32."""
    return _fp8_64((y / scale).float().double(), dt)


def _ckpt_64(x):
    """What the checkpoint of a bf16 matrix stands for."""
    r, c = x.shape
    v = torch.cat((x.double(), torch.zeros((r, -c % 32), dtype=torch.float64, device=x.device)), 1).reshape(r, -1, 32)
    a = v.abs().amax(2, keepdim=True)
    p = torch.exp2(torch.floor(torch.log2((a / 448).clamp(min=2.0 ** -130))) - 1)
    p = torch.where(448 * p < a, 2 * p, p)
    p = torch.where(448 * p < a, 2 * p, p).clamp(min=2.0 ** -127)
    return (_fp8_64(v / p, E4) * p).reshape(r, -1)[:, :c]


def _half(y):
    """Rounded to bf16, in 64 bits."""
    return y.to(torch.bfloat16).double()


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.dtype != torch.int32}
    top = lambda t: t.abs().max().reshape(1)  # noqa: E731
    if op == "linear":
        z = torch.mm(d["a"], d["b"].t()) * d["sa"] * d["sb"]
        if s["bias_t"] is not None:
            z = z + d["bias_t"]
        y = _gelu_64(z) if s["gelu"] else z
        if s["res"] is not None:
            y = y + d["res"]
        out = {}
        if s["out"] != "bf16":
            out["q"] = _quotient_64(_half(y), d["q_scale"], E4)
            out["amax"] = top(_half(y))
        if s["out"] != "q":
            out["y"] = y
        if s["ckpt"]:
            out["h"] = _ckpt_64(z.to(torch.bfloat16))
        return out
    if op == "grads":
        return {"dx": torch.mm(d["dy"], d["w"]) * d["sdy"] * d["sw"], "dw": torch.mm(d["dy"].t(), d["x"]) * d["sdy"] * d["sx"] + d["dw"]}
    if op in ("experts", "experts_grads"):
        cut = s["off"].tolist()
        spans = list(zip(cut[:-1], cut[1:]))
    if op == "experts":
        q = torch.empty((s["rows"], s["ffn"]), dtype=torch.float64, device="cuda")
        y = torch.empty((s["rows"], s["hidden"]), dtype=torch.float64, device="cuda")
        amax = torch.zeros(1, dtype=torch.float64, device="cuda")
        for e, (i, j) in enumerate(spans):
            if i == j:
                continue
            a = _half(_gelu_64(torch.mm(d["x"][i:j], d["w1"][e].t()) * d["sx"] * d["s1"] + d["b1"][e]))
            amax = torch.maximum(amax, top(a))
            q[i:j] = _quotient_64(a, d["q_scale"], E4)
            y[i:j] = torch.mm(q[i:j], d["w2"][e].t()) * d["q_scale"] * d["s2"]
        return {"q": q, "amax": amax, "y": y}
    if op == "experts_grads":
        dx = torch.empty((s["rows"], s["k"]), dtype=torch.float64, device="cuda")
        dw = torch.empty((s["experts"], s["n"], s["k"]), dtype=torch.float64, device="cuda")
        for e, (i, j) in enumerate(spans):
            dx[i:j] = torch.mm(d["dy"][i:j], d["w"][e]) * d["sdy"] * d["sw"]
            dw[e] = torch.mm(d["dy"][i:j].t(), d["x"][i:j]) * d["sdy"] * d["sx"]
        return {"dx": dx, "dw": dw}
    if op == "checkpoint":
        return {"y": _ckpt_64(s["x"])}
    r, c = s["rows"], s["cols"]
    scales = torch.exp2(d["h_sf"] - 127).unsqueeze(2).expand(-1, -1, 32).reshape(r, -1)[:, :c]
    g = d["dy"] * _gelu_slope_64(d["h"] * scales)
    return {"q": _quotient_64(_half(g), d["scale"], E4 if s["fmt"] == "e4" else E5), "amax": top(_half(g)), "d_bias": g.sum(0)}
