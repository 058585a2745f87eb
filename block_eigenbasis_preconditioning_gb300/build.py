"""Build the CUDA library `libdobb.so` in-tree for sm_103a.

Each translation unit under csrc/ is compiled with nvcc in parallel, then
linked into one shared library with a C ABI (include/dobb.h).  No CMake, no
torch extension machinery: the library depends only on the CUDA runtime.
Beside it lies `_lm_call.so`, a Python module of one C++ file that calls it with
tensors (csrc/lm_call.cpp), compiled against the installed PyTorch and Python, and again
when one of the two has changed.  The library neither needs it nor waits for it: without their
headers it is left out, and lm.py makes its calls through ctypes.

    python -m block_eigenbasis_preconditioning_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libdobb.so")
CALL = os.path.join(BUILD, "_lm_call.so")
CALL_FOR = os.path.join(BUILD, "_lm_call.for")  # the PyTorch and the Python that it was compiled against
CALL_SRC = os.path.join(CSRC, "lm_call.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdobb.so")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _mtime(files) -> float:
    return max(os.path.getmtime(f) for f in [*files, os.path.join(INCLUDE, "dobb.h")])


def _newer(target: str, files) -> bool:
    return os.path.exists(target) and os.path.getmtime(target) >= _mtime(files)


def _library_is_fresh() -> bool:
    return _newer(LIB, sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")])


def _compile(nvcc: str, src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


class NoHeaders(RuntimeError):
    """PyTorch or Python cannot be compiled against here."""


def _call_includes():
    """The include folders of PyTorch, Python and CUDA."""
    try:
        import torch
    except ImportError as e:
        raise NoHeaders(f"PyTorch is not installed ({e})") from e
    if not torch.version.cuda:
        raise NoHeaders("PyTorch was built without CUDA")
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    python = sysconfig.get_paths()["include"]
    for f in (os.path.join(python, "Python.h"), os.path.join(base, "ATen", "core", "Tensor.h")):
        if not os.path.exists(f):
            raise NoHeaders(f"{f} does not exist")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    return [python, base, os.path.join(base, "torch", "csrc", "api", "include"), cuda, INCLUDE]


def _call_is_for() -> str:
    import torch
    return f"{torch.__version__} {os.path.dirname(torch.__file__)} {torch.compiled_with_cxx11_abi()} {sys.version} {sysconfig.get_config_var('SOABI')}"


def _call_is_fresh() -> bool:
    if not _newer(CALL, [CALL_SRC]) or not os.path.exists(CALL_FOR):
        return False
    with open(CALL_FOR) as f:
        return f.read() == _call_is_for()


def _compile_call() -> str:
    inc = _call_includes()
    import torch
    obj = os.path.join(BUILD, "lm_call.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *(f"-I{i}" for i in inc),
          "-c", CALL_SRC, "-o", obj], "g++ lm_call.cpp")
    return obj


def _link_call(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALL + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-l:libdobb.so", "-Wl,-rpath,$ORIGIN", f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10",
          "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"], "link of _lm_call.so")
    os.replace(tmp, CALL)
    with open(CALL_FOR, "w") as f:
        f.write(_call_is_for())


def build_library(force: bool = False, extra_flags=None) -> str:
    """Compile (if stale) and return the path of libdobb.so; needs nvcc alone."""
    extra = list(extra_flags or [])
    if not force and not extra and _library_is_fresh():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(nvcc, s, extra), srcs))
    tmp = LIB + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-Xlinker", "-soname=libdobb.so", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB)
    return LIB


def build_call(force: bool = False) -> str:
    """Compile (if stale) and return the path of _lm_call.so, beside a built library.
    NoHeaders where that is not possible here."""
    _call_includes()
    if force or not _call_is_fresh():
        _link_call(_compile_call())
    return CALL


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile (if stale) both, and return the path of libdobb.so."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        # (compiled while nvcc works, linked after the library)
        obj = ex.submit(lambda: None if not force and _call_is_fresh() else _compile_call())
        build_library(force, extra_flags)
    try:
        if obj.result():
            _link_call(obj.result())
    except NoHeaders as e:
        print(f"_lm_call.so is left out: {e}")
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
