"""The FP8 products, the 8-bit checkpoint and the GELU's derivative in 64 bits, for the tests: plain torch on whatever
device the inputs are on, written from the definitions in include/fp8q.h."""
import math

import numpy as np
import torch

E4M3FN, E5M2 = 0, 1
DTYPE = {E4M3FN: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
TOP = {E4M3FN: 448.0, E5M2: 57344.0}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def values(codes, fmt):
    """float64 values of FP8 codes (uint8)."""
    return codes.view(DTYPE[fmt]).float().double()


def random_codes(shape, fmt, g, spread=2.0):
    """Codes of normal values, of every exponent where ``spread`` is large; none of them NaN or infinite."""
    x = torch.randn(shape, generator=g, device=g.device)
    x = x * torch.exp2((torch.rand(shape, generator=g, device=g.device) - 0.5) * spread)
    return x.clamp(-TOP[fmt], TOP[fmt]).to(DTYPE[fmt]).view(torch.uint8)


def gelu(x):
    x = x.double()
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


def gelu_slope(x):
    x = x.double()
    c = math.sqrt(2 / math.pi)
    y = x.clamp(-30, 30)  # beyond, the derivative is 0 or 1 in 64 bits
    t = torch.tanh(c * (y + 0.044715 * y ** 3))
    s = 0.5 * (1 + t) + 0.5 * y * (1 - t * t) * c * (1 + 3 * 0.044715 * y * y)
    return torch.where(x.isnan(), x, s)


def checkpoint(bits):
    """(codes, scale bytes, values in float64) of a bf16 matrix given by its bits (numpy uint16 [rows, cols]).  The codes
    come from a search over e4m3's values, the scale from a search over powers of two.  Codes of blocks with a NaN
    are 0 here (they are free)."""
    r, c = bits.shape
    x = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    nb = -(-c // 32)
    v = np.zeros((r, nb * 32))
    v[:, :c] = x
    v = v.reshape(r, nb, 32)
    nan = np.isnan(v).any(-1)
    top = (2.0 - 2.0 ** -7) * 2.0 ** 127  # the largest finite bf16
    a = np.minimum(np.nan_to_num(np.abs(v), nan=0.0, posinf=top).max(-1), top)
    powers = np.exp2(np.arange(-127, 128).astype(np.float64))
    e = np.searchsorted(448 * powers, a, side="left") - 127  # the least with a <= 448 * 2^e
    grid = np.array(sorted({(m / 8 if ex == 0 else 1 + m / 8) * 2.0 ** (max(ex, 1) - 7) for ex in range(16) for m in range(8)
                            if not (ex == 15 and m == 7)}))
    with np.errstate(invalid="ignore"):
        q = np.where(nan[..., None], 0.0, v / np.exp2(e.astype(np.float64))[..., None])
    m = np.minimum(np.abs(q), 448.0)
    hi = np.clip(np.searchsorted(grid, m), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - grid[lo], grid[hi] - m
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)  # the grid's index is the code
    out = code.astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 7)
    with np.errstate(over="ignore"):
        val = np.copysign(grid[code], q) * np.exp2(e.astype(np.float64))[..., None]
    val = np.where(np.abs(val) >= 2.0 ** 128, np.copysign(np.inf, val), val)
    val = np.where(nan[..., None], np.nan, val)
    sf = np.where(nan, 255, e + 127).astype(np.uint8)
    flat = lambda t: t.reshape(r, nb * 32)[:, :c]  # noqa: E731
    return flat(out), sf, flat(val), flat(np.broadcast_to(nan[..., None], v.shape))


def sum_bound(a, b):
    """How far binary32 sums of exact products, in any order, may be off: [m, n] for float64 a [m, k] and b [n, k].  Each of
    k additions rounds (or truncates) to a step of 2^-23 of what is held."""
    return (a.abs() @ b.abs().t()) * ((a.shape[1] + 2) * 2.0 ** -23)
