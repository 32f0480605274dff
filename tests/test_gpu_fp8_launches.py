"""The FP8 products, checkpoints and gradients: launches a call makes, their first use in a process captured, calls between
kernels that take tensor memory themselves, and from Python threads."""
import ctypes
import os
import subprocess
import sys
import threading
import time

import pytest
import torch

import fp8_reference as R
from conftest import ROOT
from quantize_amax_scaling_gb300 import fp8q
from test_gpu_binding_threads import SLOW
from test_gpu_fp8_matmul import gen
from test_gpu_launch_count import _graph_nodes
from test_gpu_tensor_memory_order import neighbour  # noqa: F401

pytestmark = pytest.mark.gpu


def calls(dev, m, n, k):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    f32 = lambda *s: torch.ones(s, device=dev)  # noqa: E731
    a, b, w, off = u8(m, k), u8(n, k), u8(3, n, k), torch.tensor([0, m // 2, m // 2, m], dtype=torch.int32, device=dev)
    q, one, amax, (h, hs) = u8(m, n), f32(1), f32(1), fp8q.checkpoint_empty(m, n)
    at, bt, dw, y, bias = u8(k, (m + 15) // 16 * 16)[:, :m], u8(k, n), f32(3, k, n), bf(m, n), f32(n)
    space = torch.empty(fp8q.gelu_backward_workspace(m, n) + 16, dtype=torch.uint8, device=dev)
    sums = 2 if fp8q.gelu_backward_workspace(m, n) else 1
    return {
        "product": (lambda: fp8q.fp8q_matmul(a, b, y), 1, 1),
        "whole epilogue": (lambda: fp8q.fp8q_matmul(a, b, y, bias=bias, act=1, residual=y, q=q, q_scale=one, amax=amax, h=h, h_sf=hs), 1, 1),
        "transposed": (lambda: fp8q.fp8q_matmul(at, bt, y, a_trans=True, b_trans=True), 1, 1),
        "product of nothing": (lambda: fp8q.fp8q_matmul(a[:, :0].contiguous(), b[:, :0].contiguous(), y, bias=bias), 1, 1),
        "grouped": (lambda: fp8q.fp8q_grouped_matmul(a, w, off, y), 1, 1),
        "weight gradients": (lambda: fp8q.fp8q_grouped_weight_gradient(a, y.view(torch.uint8)[:, :n].contiguous(), off, dw), 1, None),
        "checkpoint": (lambda: fp8q.fp8q_checkpoint_quantize(y, h, hs), 1, 1),
        "and back": (lambda: fp8q.fp8q_checkpoint_dequantize(h, hs, y), 1, 1),
        "through the GELU": (lambda: fp8q.fp8q_gelu_backward_quantize_amax(y, h, hs, q, 1, one, amax), 1, 1),
        "with the bias": (lambda: fp8q.fp8q_gelu_backward_quantize_amax(y, h, hs, q, 1, one, amax, d_bias=bias, workspace=space), sums, sums),
    }


@pytest.mark.parametrize("m,n,k", [(1, 4096, 512), (70, 208, 2064), (2560, 2304, 1056), (33, 64, 16384)])
def test_launches(m, n, k):
    dev = torch.device("cuda:0")
    s = torch.cuda.Stream()
    todo = calls(dev, m, n, k)
    torch.cuda.synchronize()
    for name, (fn, kernels, nodes) in todo.items():
        if nodes is not None:
            assert _graph_nodes(fn, s) == (kernels, nodes), name


FIRST = r"""
import torch
from quantize_amax_scaling_gb300 import fp8q
dev = torch.device("cuda:0")
m, n, k = %d, %d, %d
g = torch.Generator(device=dev)
g.manual_seed(5)
f = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.float8_e4m3fn).view(torch.uint8)
x, w, off = f(m, k), f(3, n, k), torch.tensor([0, m // 3, m // 3, m], dtype=torch.int32, device=dev)
one = torch.ones(1, device=dev)

def room():
    o = {"y": torch.zeros(m, n, dtype=torch.bfloat16, device=dev), "q": torch.zeros(m, n, dtype=torch.uint8, device=dev), "amax": torch.zeros(2, device=dev)}
    o |= {"h": torch.zeros(m, n, dtype=torch.uint8, device=dev), "s": torch.zeros(m, (n + 31) // 32, dtype=torch.uint8, device=dev)}
    o |= {"z": torch.zeros_like(o["y"]), "d": torch.zeros_like(o["q"]), "b": torch.zeros(n, device=dev), "dw": torch.zeros(3, k, n, device=dev)}
    o |= {"space": torch.zeros(1 << 24, dtype=torch.uint8, device=dev), "gy": torch.zeros_like(o["y"]), "dx": torch.zeros(m, k, device=dev)}
    return o

def step(o):
    fp8q.fp8q_matmul(x, w[0], o["y"], act=1, q=o["q"], q_scale=one, amax=o["amax"][:1], h=o["h"], h_sf=o["s"])
    fp8q.fp8q_checkpoint_dequantize(o["h"], o["s"], o["z"])
    fp8q.fp8q_gelu_backward_quantize_amax(o["y"], o["h"], o["s"], o["d"], 1, one, o["amax"][1:], d_bias=o["b"], workspace=o["space"])
    fp8q.fp8q_grouped_matmul(x, w, off, o["gy"])
    fp8q.fp8q_matmul(o["d"], w[1], o["dx"], 1, 0, b_trans=True)
    fp8q.fp8q_grouped_weight_gradient(x, o["q"], off, o["dw"], 0, 0)

first, eager = room(), room()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr, stream=torch.cuda.Stream()):
    step(first)
gr.replay()
torch.cuda.synchronize()
step(eager)
torch.cuda.synchronize()
assert eager["dw"].any() and all(torch.equal(first[i], eager[i]) for i in eager if i != "space")
gr.replay()
torch.cuda.synchronize()
assert all(torch.equal(first[i], eager[i]) for i in eager if i != "space")
print("OK")
"""


@pytest.mark.parametrize("m,n,k", [(3, 208, 1040), (100, 208, 1040), (2560, 2304, 1056)])
def test_first_call_inside_graph_capture(m, n, k):
    """In a fresh process: shared-memory limits, tensor maps and the SM count are asked for within the capture."""
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", FIRST % (m, n, k)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout + r.stderr


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (24, 6000, 4096), (300, 520, 320), (2560, 2304, 1104)])
def test_between_neighbours(neighbour, m, n, k):  # noqa: F811
    dev = torch.device("cuda:0")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = gen(dev, k)
    a, b = R.random_codes((m, k), 0, g), R.random_codes((n, k), 0, g)
    want = torch.empty((m, n), device=dev)
    fp8q.fp8q_matmul(a, b, want)
    got = [torch.zeros_like(want) for _ in range(3)]
    count = torch.zeros(1, dtype=torch.int64, device=dev)
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    for d in got:
        assert neighbour(0, sms, count.data_ptr(), side.cuda_stream) == 0
        fp8q.fp8q_matmul(a, b, d, stream=side)
        assert neighbour(1, sms, count.data_ptr(), side.cuda_stream) == 0
        fp8q.fp8q_matmul(a, b, d, stream=side)
    side.synchronize()
    assert int(count) == 6 * sms
    for d in got:
        assert torch.equal(d, want)


@pytest.fixture
def slow_calls(tmp_path):
    (tmp_path / "slow.c").write_text(SLOW)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "slow.so"), str(tmp_path / "slow.c")], check=True)
    at = ctypes.cast(ctypes.CDLL(str(tmp_path / "slow.so")).slow, ctypes.c_void_p).value
    fp8q._native().bind_products(*[at] * 7)
    yield
    fp8q._binding = None
    fp8q._native()  # the library's own again


@pytest.mark.parametrize("which", range(6))
def test_other_threads_run_while_a_launch_waits(slow_calls, which):
    dev = torch.device("cuda:0")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)  # noqa: E731
    x, d, off, (h, s) = u8(8, 64), torch.zeros((8, 8), device=dev), torch.zeros(2, dtype=torch.int32, device=dev), (u8(8, 64), u8(8, 2))
    y = torch.zeros((8, 64), dtype=torch.bfloat16, device=dev)
    call = [lambda: fp8q.fp8q_matmul(x, x, d), lambda: fp8q.fp8q_grouped_matmul(x, x[None], off, d),
            lambda: fp8q.fp8q_grouped_weight_gradient(x, x, off, torch.zeros((1, 64, 64), device=dev)),
            lambda: fp8q.fp8q_checkpoint_quantize(y, h, s), lambda: fp8q.fp8q_checkpoint_dequantize(h, s, y),
            lambda: fp8q.fp8q_gelu_backward_quantize_amax(y, h, s, d_x=y.clone())][which]
    torch.cuda.synchronize()
    seen, stop = [0], threading.Event()

    def other():
        while not stop.is_set():
            seen[0] += 1
            time.sleep(0.002)

    t = threading.Thread(target=other)
    t.start()
    time.sleep(0.05)
    before, began = seen[0], time.monotonic()
    call()
    took, after = time.monotonic() - began, seen[0]
    stop.set()
    t.join()
    assert took >= 0.29 and after - before >= 20  # of about 150


def test_first_call_of_a_thread():
    """A thread whose first call of CUDA is a product's: it has no context of its own yet."""
    dev = torch.device("cuda:0")
    a, b = torch.full((300, 256), 0x38, dtype=torch.uint8, device=dev), torch.full((300, 256), 0x38, dtype=torch.uint8, device=dev)
    q, s = fp8q.fp4_empty(300, 256, fp8q.MXFP4)
    q.fill_(0x22)
    s.fill_(127)
    d, d4, stream = torch.zeros((300, 300), device=dev), torch.zeros((300, 300), device=dev), torch.cuda.Stream()
    fp8q.fp8q_matmul(a, b, d)
    fp8q.fp8q_fp4_matmul(q, s, q, s, d4, 256, fp8q.MXFP4)
    d.zero_(), d4.zero_()
    torch.cuda.synchronize()
    for call in (lambda: fp8q.fp8q_matmul(a, b, d, stream=stream), lambda: fp8q.fp8q_fp4_matmul(q, s, q, s, d4, 256, fp8q.MXFP4, stream=stream)):
        failed = []

        def work():
            try:
                call()
            except fp8q.Fp8qError as e:
                failed.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        assert not failed
    torch.cuda.synchronize()
    assert (d == 256).all() and (d4 == 256).all()


def test_calls_of_several_threads():
    dev = torch.device("cuda:0")
    g = gen(dev, 2)
    a, b = R.random_codes((40, 256), 0, g), R.random_codes((300, 256), 0, g)
    want = torch.empty((40, 300), device=dev)
    fp8q.fp8q_matmul(a, b, want)
    torch.cuda.synchronize()
    got = [[torch.zeros_like(want) for _ in range(50)] for _ in range(4)]

    def work(ds):
        s = torch.cuda.Stream()
        for d in ds:
            fp8q.fp8q_matmul(a, b, d, stream=s)
        s.synchronize()

    ts = [threading.Thread(target=work, args=(ds,)) for ds in got]
    torch.cuda.synchronize()
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert all(torch.equal(d, want) for ds in got for d in ds)
