"""What build() makes and needs, on a copy of the package with tools that only write their output file: the library with
nvcc alone, and beside it the binding where torch is there."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

PKG = "quantize_amax_scaling_gb300"
TOOL = """#!{python}
import sys
open({log!r}, "a").write({name!r} + "\\n")
if {fails}:
    sys.exit(1)
open(sys.argv[sys.argv.index("-o") + 1], "w").close()
"""


@pytest.fixture
def copy(tmp_path):
    """A copy of the sources, tools of its own, and run(code): what code prints there, and the tools it called."""
    root = tmp_path / "root"
    shutil.copytree(os.path.join(ROOT, PKG), root / PKG, ignore=shutil.ignore_patterns("*.so", "_build", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), root / "include")
    log = tmp_path / "log"

    def tool(path, fails=False):
        path.parent.mkdir(parents=True, exist_ok=True)
        path.write_text(TOOL.format(python=sys.executable, log=str(log), name=path.name, fails=fails))
        path.chmod(0o755)

    tool(tmp_path / "cuda" / "bin" / "nvcc")
    tool(tmp_path / "bin" / "g++")

    def run(code):
        log.write_text("")
        env = dict(os.environ, CUDA_HOME=str(tmp_path / "cuda"), PATH=f"{tmp_path / 'bin'}{os.pathsep}{os.environ['PATH']}")
        r = subprocess.run([sys.executable, "-c", code], cwd=root, env=env, capture_output=True, text=True, timeout=300)
        return r, sorted(log.read_text().split())

    run.root, run.tool, run.path = root / PKG, tool, tmp_path
    return run


BUILD = f"from {PKG} import build; print(build.build())"
UNITS = 7


def test_the_library_needs_no_torch(copy):
    r, tools = copy("import sys; sys.modules['torch'] = None\n" + BUILD)
    assert r.returncode == 0 and r.stdout.strip() == str(copy.root / "libfp8q.so"), r.stdout + r.stderr
    assert tools == ["nvcc"] * (UNITS + 1) and (copy.root / "libfp8q.so").exists() and not (copy.root / "_binding.so").exists()
    # torch there later: the binding alone
    r, tools = copy(BUILD)
    assert r.returncode == 0 and tools == ["g++"] and (copy.root / "_binding.so").exists(), r.stdout + r.stderr
    r, tools = copy(BUILD)
    assert r.returncode == 0 and tools == []


def test_a_binding_that_does_not_compile_is_an_error_but_leaves_the_library(copy):
    copy.tool(copy.path / "bin" / "g++", fails=True)
    r, tools = copy(BUILD)
    assert r.returncode != 0 and "g++" in r.stderr
    assert (copy.root / "libfp8q.so").exists() and not (copy.root / "_binding.so").exists()


def test_each_is_made_again_for_its_own_sources(copy):
    r, tools = copy(BUILD)
    assert r.returncode == 0 and tools == ["g++"] + ["nvcc"] * (UNITS + 1), r.stdout + r.stderr
    later = os.path.getmtime(copy.root / "libfp8q.so") + 10
    os.utime(copy.root / "csrc" / "binding.cpp", (later, later))
    assert copy(BUILD)[1] == ["g++"]
    os.utime(copy.root / "csrc" / "binding.cpp", (1, 1))
    for so in ("libfp8q.so", "_binding.so"):
        os.utime(copy.root / so, (later, later))
    os.utime(copy.root / "csrc" / "tcgen05.cuh", (later + 10, later + 10))
    assert copy(BUILD)[1] == ["nvcc"] * (UNITS + 1)


def test_a_binding_of_another_torch_is_refused_and_made_again(copy):
    r, tools = copy(BUILD)
    assert r.returncode == 0 and tools == ["g++"] + ["nvcc"] * (UNITS + 1), r.stdout + r.stderr
    load = f"""
import types
from {PKG} import fp8q
fp8q.lib = types.SimpleNamespace
fp8q._native()
"""
    other = "import torch; torch.__version__ = '1.2.3'\n"
    r, _ = copy(other + load)  # before it is loaded: its symbols or layouts may be other ones
    assert r.returncode != 0 and "made for" in r.stderr and "torch 1.2.3" in r.stderr and "build" in r.stderr, r.stderr
    assert copy(other + BUILD)[1] == ["g++"]
    assert copy(other + BUILD)[1] == []
    r, _ = copy(load)
    assert r.returncode != 0 and "made for" in r.stderr and "torch 1.2.3" in r.stderr
    assert copy(BUILD)[1] == ["g++"]
    os.remove(copy.root / "_binding.so")
    r, _ = copy(load)
    assert r.returncode != 0 and "made for nothing yet" in r.stderr
