"""The 4-bit and residual-norm calls from Python threads: a call that has to wait for room in its stream's queue keeps no
other thread from running (as the ctypes calls do not), and calls from several threads at a time give what each
gives alone."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

import fp4_reference as R
from quantize_amax_scaling_gb300 import fp8q

pytestmark = pytest.mark.gpu

# stands in for every entry point, as one whose launch has to wait
SLOW = """
#include <time.h>
int slow(void) {
    const struct timespec t = {0, 300000000};
    nanosleep(&t, 0);
    return 0;
}
"""


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


@pytest.fixture
def slow_calls(tmp_path):
    (tmp_path / "slow.c").write_text(SLOW)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "slow.so"), str(tmp_path / "slow.c")], check=True)
    at = ctypes.cast(ctypes.CDLL(str(tmp_path / "slow.so")).slow, ctypes.c_void_p).value
    fp8q._native().bind(*[at] * 6)
    yield
    fp8q._binding = None
    fp8q._native()  # the library's own again


def calls(dev, rows=8, H=64, fmt=R.NVFP4):
    bf = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    x, w, r = bf(rows, H), torch.ones(H, device=dev), torch.ones(rows, device=dev)
    q, sf = fp8q.fp4_empty(rows, H, fmt)
    space = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    return [lambda: fp8q.fp8q_fp4_quantize_amax(x, q, sf, fmt),
            lambda: fp8q.fp8q_fp4_dequantize(q, sf, x, fmt),
            lambda: fp8q.fp8q_fp4_matmul(q, sf, q, sf, bf(rows, rows), H, fmt),
            lambda: fp8q.fp8q_residual_norm_quantize_amax(x, x, pre_weight=w, h=bf(rows, H)),
            lambda: fp8q.fp8q_residual_norm_backward(x, x, x, r, w, bf(rows, H), w, workspace=space)]


@pytest.mark.parametrize("which", range(5))
def test_other_threads_run_while_a_launch_waits(dev, slow_calls, which):
    call = calls(dev)[which]
    torch.cuda.synchronize()
    seen, stop = [0], threading.Event()

    def count():
        while not stop.is_set():
            seen[0] += 1
            time.sleep(0.002)

    t = threading.Thread(target=count)
    t.start()
    try:
        before = seen[0]
        call()  # 0.3 s
        during = seen[0] - before
    finally:
        stop.set()
        t.join()
    assert during >= 10, during


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
def test_calls_from_several_threads(dev, fmt):
    """Each thread its own stream and buffers, the same weight: quantize, multiply, norm."""
    m, n, k, each = 70, 208, 320, 40
    g = torch.Generator(device=dev)
    g.manual_seed(fmt)
    f = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    w = fp8q.fp4_empty(n, k, fmt)
    fp8q.fp8q_fp4_quantize_amax(f(n, k).bfloat16(), *w, fmt)
    ins = [(f(m, k).bfloat16(), f(m, n).bfloat16(), 1 + 0.1 * f(n)) for _ in range(4)]

    def step(x, res, pre, o, stream=None):
        fp8q.fp8q_fp4_quantize_amax(x, o["q"], o["sf"], fmt, stream=stream)
        fp8q.fp8q_fp4_matmul(o["q"], o["sf"], *w, o["y"], k, fmt, stream=stream)
        fp8q.fp8q_residual_norm_quantize_amax(res, o["ro"], block=o["y"], pre_weight=pre, h=o["h"], stream=stream)

    def room():
        q, sf = fp8q.fp4_empty(m, k, fmt)
        sf.zero_()
        return {"q": q, "sf": sf, **{c: torch.zeros(m, n, dtype=torch.bfloat16, device=dev) for c in ("y", "ro", "h")}}

    want = [room() for _ in ins]
    for i, o in zip(ins, want):
        step(*i, o)
    got = [room() for _ in ins]
    streams = [torch.cuda.Stream(dev) for _ in ins]
    torch.cuda.synchronize()
    wrong = []

    def work(j):
        try:
            for _ in range(each):
                step(*ins[j], got[j], stream=streams[j])
            streams[j].synchronize()
        except Exception as e:  # shown below
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(ins))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    for a, b in zip(want, got):
        assert all(torch.equal(a[c], b[c]) for c in a)
