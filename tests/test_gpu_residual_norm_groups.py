"""A gate that all rows share, said by the largest rows_per_gate there is: the same as by the number of rows."""
import ctypes

import pytest
import torch

from quantize_amax_scaling_gb300 import fp8q
from test_gpu_residual_norm import forward, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


@pytest.mark.parametrize("per", [2 ** 63 - 1, 2 ** 63 - 700, 2 ** 62, 2 ** 32 + 1])
@pytest.mark.parametrize("rows,H", [(1, 64), (2, 1040), (700, 1040), (9, 8208)])
def test_all_rows(dev, rows, H, per):
    d = make(rows, H, max(rows, 2), "f32", rows, dev)
    o = forward(d, rows, H, max(rows, 2), 0.7, 1e-6, dev=dev)
    p = forward(d, rows, H, per, 0.7, 1e-6, dev=dev)
    assert all(torch.equal(o[k], p[k]) for k in o)
    bf = lambda: torch.full((rows, H), 7.0, dtype=torch.bfloat16, device=dev)  # noqa: E731
    dro, dh = d["residual"], d["block"]

    def args(per):
        out = {"d_residual": bf(), "d_pre_weight": torch.full((H,), 7.0, device=dev), "d_block": bf(),
               "d_post_weight": torch.full((H,), 7.0, device=dev), "d_gate": torch.full_like(d["gate"], 7.0)}
        return out, torch.empty(fp8q.residual_norm_backward_workspace(rows, H, per), dtype=torch.uint8, device=dev)

    got = []
    for n in (max(rows, 2), per):
        out, space = args(n)
        fp8q.fp8q_residual_norm_backward(dro, dh, o["ro"], o["rstd_pre"], d["pre"], out["d_residual"], out["d_pre_weight"], block=d["block"],
                                         rstd_post=o["rstd_post"], post_weight=d["post"], gate=d["gate"], rows_per_gate=n, alpha=0.7,
                                         d_block=out["d_block"], d_post_weight=out["d_post_weight"], d_gate=out["d_gate"], workspace=space)
        got.append(out)
    out, space = args(per)  # the C call, without the binding's own checks
    ptr = lambda t: t.data_ptr()  # noqa: E731
    c = fp8q.ResidualNormGrad(rows=rows, hidden=H, gate_is_bf16=0, d_residual_out=ptr(dro), d_h=ptr(dh), residual_out=ptr(o["ro"]),
                              rstd_pre=ptr(o["rstd_pre"]), pre_weight=ptr(d["pre"]), block=ptr(d["block"]), rstd_post=ptr(o["rstd_post"]),
                              post_weight=ptr(d["post"]), gate=ptr(d["gate"]), rows_per_gate=per, alpha=0.7, workspace=ptr(space),
                              workspace_bytes=space.numel(), **{k: ptr(t) for k, t in out.items()})
    assert fp8q.lib().fp8q_residual_norm_backward(ctypes.byref(c), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for k, t in got[0].items():
        assert torch.equal(got[1][k], t) and torch.equal(out[k], t), k
