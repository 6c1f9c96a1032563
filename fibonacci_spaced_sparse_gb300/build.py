"""Build libsfa.so in-tree with nvcc for sm_103a (GB300), and the native half
of the Python binding with g++.

Each .cu file under csrc/ is compiled in parallel into an object, then they
are linked into ``fibonacci_spaced_sparse_gb300/_build/libsfa.so``;
csrc/bind.cpp becomes ``_build/_sfa_bind.so``, which uses libsfa.so and the
installed torch.  Either is skipped when it is newer than its sources and
headers, the binding if the same torch and Python are there as well.

libsfa.so, the C ABI, needs nvcc alone: where torch is not installed the binding
is left out, and ``--no-binding`` leaves it out anywhere.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libsfa.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(BUILD, "_sfa_bind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def lib_up_to_date() -> bool:
    return _newer(LIB, sources() + _headers())


def binding_up_to_date() -> bool:
    return _newer(BIND, [BIND_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))) and built_for(BIND) == binding_key()


def binding_key() -> str:
    """What a binding is built for: the installed torch and the interpreter."""
    import torch
    return (f"torch {torch.__version__} in {os.path.dirname(torch.__file__)}, "
            f"Python {sys.version_info.major}.{sys.version_info.minor}")


def built_for(path: str) -> str:
    """The key that the binding at ``path`` was built with, kept beside it."""
    try:
        with open(path + ".key") as f:
            return f.read()
    except OSError:
        return ""


def _compile_bind() -> str:
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           cuda, sysconfig.get_paths()["include"]]
    obj = os.path.join(BUILD, "obj", "bind.cpp.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{p}" for p in inc),
           "-c", BIND_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BIND_SRC}:\n{r.stderr}")
    return obj


def _link_bind(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + f".{os.getpid()}.tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-l:libsfa.so", f"-L{lib}", "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    if os.path.exists(BIND + ".key"):
        os.remove(BIND + ".key")
    os.replace(tmp, BIND)
    with open(BIND + ".key", "w") as f:
        f.write(binding_key())


def build(force: bool = False, ptxas_info: bool = False, binding: bool | None = None) -> str:
    """Compile and link libsfa.so and the binding (``binding``: None builds it
    where torch is installed); returns libsfa.so's path.  libsfa.so is there
    even when the binding fails to build."""
    if binding is None:
        binding = importlib.util.find_spec("torch") is not None
    force = force or ptxas_info
    with_lib = force or not lib_up_to_date()
    with_bind = binding and (force or not binding_up_to_date())
    if not with_lib and not with_bind:
        return LIB
    os.makedirs(os.path.join(BUILD, "obj"), exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, "obj", os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        bind_obj = ex.submit(_compile_bind) if with_bind else None  # the slowest one: first
        objs = list(ex.map(compile_one, sources())) if with_lib else []
    if with_lib:
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    if with_bind:
        _link_bind(bind_obj.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_info="--ptxas" in sys.argv,
                binding=False if "--no-binding" in sys.argv else None))
