"""The microscaled 4-bit formats written out in numpy float64, from their definitions: what the
kernels of the packed 4-bit operands are compared with.  Quotients that the definition rounds to
binary32 are divided in float64 first; for two binary32 numbers that double rounding is harmless
(53 >= 2 * 24 + 2 bits)."""
import numpy as np

MXFP4, NVFP4 = 2, 3
BLOCK = {MXFP4: 32, NVFP4: 16}
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
VALUE = np.concatenate([GRID, -GRID])


def bf16_to_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_values():
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v + [np.nan])


E4M3 = e4m3_values()


def nearest_even(v, grid):
    """Index of the nearest entry of the ascending `grid` to v >= 0, ties to the even index, held at the last."""
    v = np.minimum(v, grid[-1])
    hi = np.clip(np.searchsorted(grid, v, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantize(bits, fmt, scale=None):
    """bits: bf16 [r, c].  Codes [r, c], block scale bytes [r, blocks], and which blocks are NaN."""
    x = bf16_to_f64(bits)
    r, c = x.shape
    b = BLOCK[fmt]
    nb = -(-c // b)
    v = np.zeros((r, nb * b))
    v[:, :c] = x
    v = v.reshape(r, nb, b)
    nan = np.isnan(v).any(2)
    a = np.where(np.isnan(v), 0, np.abs(v)).max(2)
    with np.errstate(all="ignore"):
        if fmt == MXFP4:
            top = np.minimum(a, bf16_to_f64([0x7F7F])[0])
            e = np.where(top > 0, np.frexp(top)[1] - 3, -127)
            e = np.maximum(e, -127)
            sf = np.where(nan, 255, e + 127).astype(np.uint8)
            u = v / np.ldexp(1.0, e)[..., None]
        else:
            s = np.float32(1.0 if scale is None else scale)
            s6 = np.float32(s * np.float32(6))
            good = bool(s6 > 0) and bool(np.isfinite(s6))
            quo = (a / np.float64(s6)).astype(np.float32).astype(np.float64) if good else np.zeros_like(a)
            sf = nearest_even(quo, E4M3[:127]).astype(np.uint8)
            if not good:
                sf = np.where(a != 0, 127, 0).astype(np.uint8)
                nan = nan | (a != 0)
            sf = np.where(nan, 127, sf)
            sf = np.where((a == 0) & ~nan, 0, sf).astype(np.uint8)
            d = (np.where(sf == 127, 0, E4M3[sf]) * np.float64(s) if good else np.zeros_like(a))
            d = d.astype(np.float32).astype(np.float64)[..., None]
            u = np.where(d > 0, np.where(np.isinf(v), v, v / np.where(d > 0, d, 1)), 0)
            u = u.astype(np.float32).astype(np.float64)
    u = np.where(np.isnan(u), 0, u)
    codes = nearest_even(np.abs(u), GRID).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 3)
    return codes.reshape(r, -1)[:, :c], sf, nan


def sf_values(sf, fmt):
    if fmt == MXFP4:
        return np.where(sf == 255, np.nan, np.ldexp(1.0, sf.astype(np.int64) - 127))
    return np.where(sf & 0x80, -1.0, 1.0) * E4M3[sf & 0x7F]


def values(codes, sf, fmt, scale=None):
    """float64 [r, c]: code * block scale * scale, unrounded."""
    c = codes.shape[1]
    s = np.repeat(sf_values(sf, fmt), BLOCK[fmt], axis=1)[:, :c]
    return VALUE[codes] * s * (1.0 if scale is None else np.float64(np.float32(scale)))


def sf_place(r, nb):
    i, j = np.arange(r)[:, None], np.arange(nb)[None, :]
    return ((i // 128) * (-(-nb // 4)) + j // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4


def pack(codes, sf):
    """Packed codes and scales; bytes of the scales that belong to no row come out as 0xEE."""
    r, c = codes.shape
    full = np.zeros((r, 32 * (-(-c // 32))), np.uint8)
    full[:, :c] = codes
    nb4 = 4 * (-(-sf.shape[1] // 4))
    out = np.full(-(-r // 128) * (nb4 // 4) * 512, 0xEE, np.uint8)
    out[sf_place(r, nb4)] = 0
    out[sf_place(r, sf.shape[1])] = sf
    return full[:, 0::2] | (full[:, 1::2] << 4), out


def unpack(q, s, r, c, fmt):
    q = np.asarray(q).reshape(r, -1)
    full = np.empty((r, q.shape[1] * 2), np.uint8)
    full[:, 0::2], full[:, 1::2] = q & 15, q >> 4
    return full[:, :c], np.asarray(s)[sf_place(r, -(-c // BLOCK[fmt]))]
