"""Sizes of packed operands and workspaces where a size is beyond what the calls take: 0, and no arithmetic that
divides by zero or leaves 64 bits on the way there."""
import ctypes
import subprocess
import sys

import pytest

from conftest import ROOT

TOP = 2 ** 31 - 1024  # the most rows and columns of an operand, the most rows of a norm


def test_operands_of_refused_sizes():
    from quantize_amax_scaling_gb300 import build, fp8q
    build.build()
    L = fp8q.lib()
    i64 = ctypes.c_int64
    L.fp8q_fp4_row_bytes.argtypes, L.fp8q_fp4_row_bytes.restype = [i64], i64
    L.fp8q_fp4_scale_bytes.argtypes, L.fp8q_fp4_scale_bytes.restype = [i64, i64, ctypes.c_int], i64
    assert L.fp8q_fp4_row_bytes(TOP) == fp8q.fp4_row_bytes(TOP)
    for fmt in (fp8q.MXFP4, fp8q.NVFP4):
        assert L.fp8q_fp4_scale_bytes(TOP, TOP, fmt) == fp8q.fp4_scale_bytes(TOP, TOP, fmt)
        for big in (TOP + 1, 2 ** 53, 2 ** 63 - 1):
            assert L.fp8q_fp4_scale_bytes(big, 64, fmt) == L.fp8q_fp4_scale_bytes(64, big, fmt) == 0
            assert L.fp8q_fp4_row_bytes(big) == 0


def test_workspace_of_refused_sizes():
    """In a process of its own: a division by zero would end it."""
    code = f"""
from quantize_amax_scaling_gb300 import build, fp8q
build.build()
w = fp8q.residual_norm_backward_workspace
assert w(5, 32768) > 0 and w({TOP}, 32768, 7) > 0
for rows, hidden in ((1, 32769), (1, 304 * 4096), (1, 304 * 4096 + 1), (1, 2 ** 31 - 1), (7, 2 ** 40), ({TOP + 1}, 64), (2 ** 63 - 1, 64)):
    for per in (0, 1, 5, 2 ** 63 - 1):
        assert w(rows, hidden, per) == 0, (rows, hidden, per)
print("OK")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("OK\n"), (r.returncode, r.stdout + r.stderr)


def test_room_of_refused_sizes():
    """fp4_empty says no before it asks for memory: of 2^53 rows of 2^15 columns both arrays' bytes are 0 modulo 2^64."""
    from quantize_amax_scaling_gb300 import build, fp8q
    build.build()
    for device in ("cuda", "cpu"):
        for rows, cols in ((2 ** 53, 2 ** 15), (TOP + 1, 16), (16, TOP + 1), (-1, 16), (16, -1)):
            for fmt in (fp8q.MXFP4, fp8q.NVFP4):
                with pytest.raises(ValueError, match="rows and cols"):
                    fp8q.fp4_empty(rows, cols, fmt, device=device)
        with pytest.raises(ValueError):
            fp8q.fp4_empty(4, 64, fp8q.E4M3FN, device=device)
