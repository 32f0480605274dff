"""Compile libfp8q.so (the CUDA kernels and their C ABI) for sm_103a, in tree.

Translation units compiled in parallel with one -gencode each, then linked; no
cmake.  The library needs nothing else.  Beside it, where torch is there, the
compiled part of the Python binding (csrc/binding.cpp, g++ against torch's
headers).  Both and their objects are written next to this file and
git-ignored.
"""
import os
import platform
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
UNITS = ["quantize.cu", "producers.cu", "scale_update.cu", "fp4_quantize.cu", "fp4_matmul.cu", "residual_norm.cu", "fp8_matmul.cu"]
SRCS = [os.path.join(CSRC, u) for u in UNITS]
DEPS = SRCS + [os.path.join(CSRC, h) for h in ("fp8q_common.cuh", "packed_f32.cuh", "quant_tile.cuh",
                                                "slot_math.cuh", "mbarrier.cuh", "fp4.cuh", "tcgen05.cuh", "checkpoint.cuh", "checkpoint_calls.cuh")] + [os.path.join(ROOT, "include", "fp8q.h")]
LIB = os.path.join(PKG, "libfp8q.so")
OBJ_DIR = os.path.join(PKG, "_build")

BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_FOR = os.path.join(OBJ_DIR, "binding_for.txt")  # the Python and torch that _binding.so was made for
BINDING_DEPS = [BINDING_SRC, os.path.join(ROOT, "include", "fp8q.h")]
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-warn-spills",
]


def nvcc_path() -> str:
    cand = [os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"]
    for c in cand:
        p = os.path.join(c, "bin", "nvcc") if c else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found (set CUDA_HOME)")
    return p


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is missing or older than its sources: libfp8q.so, and the binding's compiled part
    where torch can be imported.  Return the library's path.  The library is made whatever becomes of the binding."""
    with ThreadPoolExecutor(1) as ex:
        binding = None
        if force or not _current(BINDING, BINDING_DEPS) or binding_for() not in (None, binding_made_for()):
            binding = ex.submit(build_binding)
        if force or not _current(LIB, DEPS):
            _build_library(verbose)
        if binding is not None:
            binding.result()
    return LIB


def binding_for():
    """The running Python and torch, whose compiled interfaces the binding uses; None without torch."""
    try:
        import torch
    except ImportError:
        return None
    return f"{sys.implementation.cache_tag} ({platform.machine()}), torch {torch.__version__}"


def binding_made_for():
    """What binding_for() was when the binding was made; None if there is none."""
    try:
        with open(BINDING_FOR) as f:
            return f.read() if os.path.exists(BINDING) else None
    except OSError:
        return None


def _current(path, deps) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(p) for p in deps)


def _build_library(verbose: bool) -> None:
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = nvcc_path()
    tag = f".{os.getpid()}"

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + tag + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj, src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        return obj

    with ThreadPoolExecutor(len(SRCS)) as ex:
        objs = list(ex.map(compile_one, SRCS))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)


def build_binding():
    """Compile _binding.so (host code; g++, torch's headers) for the running Python and torch; None without torch."""
    import sysconfig

    made_for = binding_for()
    if made_for is None:
        return None
    import torch
    os.makedirs(OBJ_DIR, exist_ok=True)
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    libs = os.path.join(home, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in inc),
                    "-o", tmp, BINDING_SRC, f"-L{libs}", f"-Wl,-rpath,{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
                    "-ltorch_python"], check=True)
    if os.path.exists(BINDING_FOR):  # never beside a binding that it is not true of
        os.remove(BINDING_FOR)
    os.replace(tmp, BINDING)
    tmp = BINDING_FOR + f".tmp{os.getpid()}"
    with open(tmp, "w") as f:
        f.write(made_for)
    os.replace(tmp, BINDING_FOR)
    return BINDING


def build_variant(lib_path: str, defines) -> str:
    """Compile the same sources with extra preprocessor definitions into lib_path.

    Only tests use this: it builds libraries whose test hooks (for example
    FP8Q_TEST_LN_GIVE_UP_AT) exercise paths that correct operation never takes.
    """
    nvcc = nvcc_path()
    out_dir = os.path.dirname(os.path.abspath(lib_path))
    os.makedirs(out_dir, exist_ok=True)
    flags = [f"-D{d}" for d in defines]

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.basename(src) + ".o")
        subprocess.run([nvcc, *NVCC_FLAGS, *flags, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj, src],
                       check=True)
        return obj

    with ThreadPoolExecutor(len(SRCS)) as ex:
        objs = list(ex.map(compile_one, SRCS))
    subprocess.run([nvcc, *ARCH, "-shared", "-o", lib_path, *objs], check=True)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
