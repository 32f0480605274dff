"""The packed 4-bit operand and the residual norms on the host: the reference's own pins, the
sizes the library and the binding give, and the refusals, none of which needs a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_reference as R

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = ctypes.c_void_p(0x10000)  # never dereferenced: the calls below fail validation or are empty
ODD = ctypes.c_void_p(0x10001)
OFF8 = ctypes.c_void_p(0x10008)
OFF2 = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    from quantize_amax_scaling_gb300 import build, fp8q
    build.build()
    L = fp8q.lib()
    L.fp8q_fp4_row_bytes.argtypes = [ctypes.c_int64]
    L.fp8q_fp4_row_bytes.restype = ctypes.c_int64
    L.fp8q_fp4_scale_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    L.fp8q_fp4_scale_bytes.restype = ctypes.c_int64
    return L


def bits(x):
    return torch.tensor(x, dtype=torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_reference_rounds_to_nearest_even_code():
    # midpoints and their neighbours, by hand: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    v = np.array([0, 0.25, 0.26, 0.74, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.49, 3.5, 5, 5.01, 6, 99, np.inf])
    assert list(R.nearest_even(v, R.GRID)) == [0, 0, 1, 1, 2, 2, 3, 4, 4, 5, 5, 6, 6, 7, 7, 7, 7]
    got = torch.from_numpy(np.linspace(0, 448, 40001)).float()
    want = got.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.nearest_even(got.double().numpy(), R.E4M3[:127]), want)


def test_reference_blocks_by_hand():
    x = np.zeros((1, 40), np.float32)
    x[0, :4] = [7.5, -3.0, 0.5, 1.0]    # max 7.5: e = 2 - 2 = 0
    x[0, 33] = 48.0                      # floor(log2 48) = 5: e = 3, 48 / 8 = 6
    c, sf, nan = R.quantize(bits(x), R.MXFP4)
    assert list(sf[0]) == [127, 130] and not nan.any()
    assert list(c[0, :4]) == [7, 13, 1, 2] and c[0, 33] == 7 and not c[0, 34:].any()
    c, sf, nan = R.quantize(bits(x), R.NVFP4, 0.5)
    # 7.5 / (6 * 0.5) = 2.5, 48 / 3 = 16, zeros between
    assert list(R.sf_values(sf, R.NVFP4)[0]) == [2.5, 0, 16]
    # divided by 1.25: 6, -2.4 -> -2, 0.4 -> 0.5, 0.8 -> 1; 48 / 8 = 6
    assert list(c[0, :4]) == [7, 12, 1, 2] and c[0, 33] == 7
    x[0, 5] = np.nan
    x[0, 35] = np.inf
    c, sf, nan = R.quantize(bits(x), R.MXFP4)
    assert list(sf[0]) == [255, 252] and list(nan[0]) == [True, False] and c[0, 35] == 7 and c[0, 33] == 0
    c, sf, nan = R.quantize(bits(x), R.NVFP4, 0.5)
    assert list(sf[0]) == [127, 0, 126] and list(nan[0]) == [True, False, False] and c[0, 35] == 7


def test_pack_and_unpack_are_inverse():
    rng = np.random.RandomState(3)
    for r, c, f in ((1, 1, 2), (130, 33, 2), (5, 129, 3), (257, 64, 3)):
        codes = rng.randint(0, 16, (r, c)).astype(np.uint8)
        sf = rng.randint(0, 255, (r, -(-c // R.BLOCK[f]))).astype(np.uint8)
        q, s = R.pack(codes, sf)
        c2, s2 = R.unpack(q, s, r, c, f)
        assert np.array_equal(c2, codes) and np.array_equal(s2, sf)


def test_sizes_agree(L):
    from quantize_amax_scaling_gb300 import fp8q
    for r, c in ((1, 1), (1, 32), (1, 33), (127, 63), (128, 64), (129, 65), (128, 128), (129, 129), (4096, 16384)):
        assert L.fp8q_fp4_row_bytes(c) == fp8q.fp4_row_bytes(c)
        for f in (R.MXFP4, R.NVFP4):
            assert L.fp8q_fp4_scale_bytes(r, c, f) == fp8q.fp4_scale_bytes(r, c, f)
            q, s = R.pack(np.zeros((r, c), np.uint8), np.zeros((r, -(-c // R.BLOCK[f])), np.uint8))
            assert q.size == r * fp8q.fp4_row_bytes(c) and s.size == fp8q.fp4_scale_bytes(r, c, f)
            t, u = fp8q.fp4_empty(r, c, f, device="cpu")
            assert t.shape == (r, fp8q.fp4_row_bytes(c)) and u.numel() == s.size
    assert L.fp8q_fp4_scale_bytes(4, 4, 0) == 0
    with pytest.raises(ValueError):
        fp8q.fp4_empty(4, 4, fp8q.E4M3FN, device="cpu")


def test_quantize_refusals(L):
    f = L.fp8q_fp4_quantize_amax
    #       x  rows cols q  sf qt sft fmt scale amax stream
    good = [P, 0, 64, P, P, P, P, 3, P, P, None]

    def call(*changes):
        a = list(good)
        a[1] = 5
        for i, v in changes:
            a[i] = v
        return f(*a)

    assert f(*good) == OK and call((2, 0)) == OK          # empty
    assert call((1, -1)) == INVALID and call((2, -1)) == INVALID
    for fmt in (0, 1, 4, -1):
        assert call((7, fmt)) == INVALID
    assert call((0, None)) == INVALID and call((0, ODD)) == INVALID
    for i in (3, 4, 5, 6):                                  # half a pair
        assert call((i, None)) == INVALID
    assert call((3, None), (4, None), (5, None), (6, None)) == INVALID
    assert call((7, 2)) == INVALID                          # a tensor scale with the power-of-two format
    assert call((8, OFF2)) == INVALID and call((9, OFF2)) == INVALID
    for i in (3, 4, 5, 6):
        assert call((i, OFF8)) == UNSUPPORTED
    assert call((1, 2 ** 31)) == UNSUPPORTED and call((2, 2 ** 31)) == UNSUPPORTED


def test_dequantize_and_matmul_refusals(L):
    f = L.fp8q_fp4_dequantize
    assert f(None, None, None, 0, 7, 2, None, None) == OK
    assert f(P, P, P, 4, 7, 0, None, None) == INVALID
    assert f(P, P, P, 4, 7, 2, P, None) == INVALID
    assert f(P, P, P, -4, 7, 2, None, None) == INVALID
    assert f(None, P, P, 4, 7, 2, None, None) == INVALID
    assert f(P, P, ODD, 4, 7, 2, None, None) == INVALID
    assert f(P, OFF8, P, 4, 7, 2, None, None) == UNSUPPORTED
    m = L.fp8q_fp4_matmul
    #       a  asf b  bsf d  m  n  k  fmt out sa sb stream
    good = [P, P, P, P, P, 3, 4, 5, 3, 0, P, P, None]

    def call(*changes):
        a = list(good)
        for i, v in changes:
            a[i] = v
        return m(*a)

    assert call((5, 0)) == OK and call((6, 0)) == OK and call((5, 0), (7, 0)) == OK
    assert call((7, 0), (4, None)) == INVALID               # k == 0 writes zeros: d has to be there
    for i in (5, 6, 7):
        assert call((i, -1)) == INVALID and call((i, 2 ** 31)) == UNSUPPORTED
    assert call((8, 1)) == INVALID and call((9, 2)) == INVALID and call((8, 2)) == INVALID
    for i in (0, 1, 2, 3, 4):
        assert call((i, None)) == INVALID
    for i in (0, 1, 2, 3):
        assert call((i, OFF8)) == UNSUPPORTED
    assert call((4, ODD)) == INVALID and call((9, 1), (4, OFF2)) == INVALID and call((10, OFF2)) == INVALID


def forward_args(**changes):
    from quantize_amax_scaling_gb300.fp8q import ResidualNorm
    p = P.value
    a = dict(rows=4, hidden=64, fmt=0, residual=p, block=p, post_weight=p, gate=p, rows_per_gate=2, gate_is_bf16=0,
             alpha=1.0, eps=1e-6, pre_weight=p, residual_out=p, h=p, q=p, sf=None, scale=p, amax=p, rstd_post=p, rstd_pre=p)
    a.update(changes)
    return ResidualNorm(**a)


def test_residual_norm_refusals(L):
    def call(**c):
        return L.fp8q_residual_norm_quantize_amax(ctypes.byref(forward_args(**c)), None)

    p = P.value
    assert L.fp8q_residual_norm_quantize_amax(None, None) == INVALID
    assert call(rows=0) == OK
    for c in (dict(rows=-1), dict(hidden=0), dict(hidden=24), dict(hidden=8), dict(fmt=4), dict(residual=None),
              dict(residual_out=None), dict(block=None), dict(block=None, post_weight=None), dict(rows_per_gate=0),
              dict(pre_weight=None), dict(pre_weight=None, h=None, q=None), dict(h=None, q=None), dict(scale=None),
              dict(sf=p), dict(fmt=2), dict(fmt=3), dict(fmt=2, sf=p), dict(q=None, sf=p), dict(scale=p + 2),
              dict(amax=p + 1), dict(rstd_pre=p + 2)):
        assert call(**c) == INVALID, c
    for c in (dict(hidden=32784), dict(rows=2 ** 31), dict(residual=p + 8), dict(block=p + 8), dict(post_weight=p + 4),
              dict(gate=p + 8), dict(h=p + 2), dict(q=p + 1), dict(residual_out=p + 8), dict(pre_weight=p + 4)):
        assert call(**c) == UNSUPPORTED, c


def test_residual_norm_backward_refusals(L):
    from quantize_amax_scaling_gb300 import fp8q
    p = P.value

    def call(**changes):
        a = dict(rows=4, hidden=64, gate_is_bf16=0, d_residual_out=p, d_h=p, residual_out=p, rstd_pre=p, pre_weight=p, block=p,
                 rstd_post=p, post_weight=p, gate=p, rows_per_gate=2, alpha=1.0, d_residual=p, d_block=p, d_pre_weight=p,
                 d_post_weight=p, d_gate=p, workspace=p, workspace_bytes=1 << 20)
        a.update(changes)
        return L.fp8q_residual_norm_backward(ctypes.byref(fp8q.ResidualNormGrad(**a)), None)

    assert L.fp8q_residual_norm_backward(None, None) == INVALID
    assert call(rows=0, d_pre_weight=None, d_post_weight=None) == OK
    assert call(rows=0, d_post_weight=p + 4) == UNSUPPORTED
    for c in (dict(rows=-1), dict(hidden=24), dict(d_residual_out=None, d_h=None), dict(residual_out=None), dict(rstd_pre=None),
              dict(pre_weight=None), dict(d_h=None), dict(block=None), dict(rstd_post=None), dict(post_weight=None),
              dict(rows_per_gate=0), dict(gate=None), dict(workspace=None), dict(workspace_bytes=16), dict(rstd_pre=p + 1)):
        assert call(**c) == INVALID, c
    for c in (dict(hidden=32784), dict(rows=2 ** 31), dict(d_h=p + 8), dict(workspace=p + 8), dict(d_gate=p + 4)):
        assert call(**c) == UNSUPPORTED, c
    w = fp8q.residual_norm_backward_workspace
    assert w(0, 64) == 0 and w(1, 64) == 2 * 64 * 4 and w(1, 64, 1) == 2 * 64 * 4 and w(1, 64, 5) == 4 * 64 * 4


def test_binding_refuses_host_and_wrong_tensors():
    from quantize_amax_scaling_gb300 import fp8q
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    q, sf = fp8q.fp4_empty(4, 32, fp8q.NVFP4, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        fp8q.fp8q_fp4_quantize_amax(x, q, sf, fp8q.NVFP4)
    with pytest.raises(ValueError, match="rows, cols"):
        fp8q.fp8q_fp4_quantize_amax(x[0], q, sf, fp8q.NVFP4)
    with pytest.raises(ValueError, match="CUDA"):
        fp8q.fp8q_fp4_matmul(q, sf, q, sf, x, 32, fp8q.NVFP4)
    with pytest.raises(ValueError, match="CUDA"):
        fp8q.fp8q_residual_norm_quantize_amax(x, x)
    with pytest.raises(ValueError):
        fp8q.fp8q_residual_norm_backward(None, None, None, None, None, None, None)
