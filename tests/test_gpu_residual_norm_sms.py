"""The residual norms' grids follow the SMs that there are: one round of resident CTAs, whose strips are as long as
they have to be; and the workspace, which is sized without a device, holds the strips of every number of SMs.  With the
library built once more with its test hooks, which take the number from the environment."""
import ctypes

import pytest
import torch

from quantize_amax_scaling_gb300 import fp8q
from test_gpu_residual_norm import check_backward, check_forward, forward, make

pytestmark = pytest.mark.gpu


class KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


@pytest.fixture
def hooked(hooks_lib, monkeypatch):
    """fp8q's calls on the hooked library."""
    path = hooks_lib._name
    monkeypatch.setattr(fp8q, "LIB_PATH", path)
    monkeypatch.setattr(fp8q, "_lib", None)
    monkeypatch.setattr(fp8q, "_binding", None)
    fp8q._native()
    yield monkeypatch
    monkeypatch.undo()
    fp8q._binding = None
    fp8q._native()


def grids(fn):
    """Warps of each kernel that fn launches."""
    drv = ctypes.CDLL("libcuda.so.1")
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g, stream=s):
        fn()
    handle, n = ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t(0)
    assert drv.cuGraphGetNodes(handle, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert drv.cuGraphGetNodes(handle, nodes, ctypes.byref(n)) == 0
    out = []
    for i in range(n.value):
        p = KernelNode()
        assert drv.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(nodes[i]), ctypes.byref(p)) == 0
        out.append(p.grid[0] * p.grid[1] * p.grid[2] * p.block[0] // 32)
    return out


@pytest.mark.parametrize("sms", [4, 40, 76, 148, 152])
@pytest.mark.parametrize("rows,H", [(700, 4096), (1300, 2064), (400, 8208), (5, 32768), (3001, 64)])
def test_as_many_strips_as_sms_take(hooked, rows, H, sms):
    hooked.setenv("FP8Q_TEST_SM_COUNT", str(sms))
    dev = torch.device("cuda:0")
    d = make(rows, H, 100, "f32", 3, dev)
    o = forward(d, rows, H, 100, 0.7, 1e-6, dev=dev)
    check_forward(d, o, rows, H, 100, 0.7, 1e-6)
    check_backward(dev, rows, H, 100, "f32")  # and nothing behind the workspace
    x = [torch.empty_like(d["residual"]) for _ in range(3)]
    w = [torch.empty(H, device=dev) for _ in range(2)]
    space = torch.empty(fp8q.residual_norm_backward_workspace(rows, H, 100), dtype=torch.uint8, device=dev)
    dgate = torch.empty_like(d["gate"])
    ahead = grids(lambda: fp8q.fp8q_residual_norm_quantize_amax(d["residual"], x[0], block=d["block"], post_weight=d["post"], gate=d["gate"],
                                                                rows_per_gate=100, pre_weight=d["pre"], h=x[1]))
    back = grids(lambda: fp8q.fp8q_residual_norm_backward(d["residual"], d["block"], x[0], o["rstd_pre"], d["pre"], x[1], w[0], block=d["block"],
                                                          rstd_post=o["rstd_post"], post_weight=d["post"], gate=d["gate"], rows_per_gate=100,
                                                          d_block=x[2], d_post_weight=w[1], d_gate=dgate, workspace=space))
    # Forward an SM holds at most 24, 20 or 16 warps by the kernel's registers, 32 of the one for wide rows; backward 16 (15 of
    # five to a CTA); a row, or a cluster of CTAs of 8 warps for one, is there in any case.
    assert len(ahead) == 1 and ahead[0] <= 32 * sms, ahead
    assert len(back) == 2 and back[0] <= max(16 * sms, -(-H // 4096) * 8), back
