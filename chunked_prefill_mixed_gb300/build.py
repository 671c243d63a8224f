"""Build in-tree: libsarathi.so with nvcc for sm_103a (host planners and kernels), and the
Python side's extension module with g++ against the installed torch."""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libsarathi.so")
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("plan.cpp", "mixed_attn.cu", "noalloc.cu", "qkv_gemm.cu", "paged_plan.cpp",
                                                        "rope_append.cu", "paged_attn.cu")]
HEADERS = [os.path.join(ROOT, "include", "sarathi.h")] + [
    os.path.join(HERE, "csrc", f) for f in ("sarathi_internal.h", "paged_internal.h", "device_util.cuh")]


def calls_path() -> str:
    """Where the extension module is: named by what it is built against, so that one of
    another Python or torch is not taken for it."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "none"
    return os.path.join(HERE, f"_paged_calls.{sys.implementation.cache_tag}-torch{torch}.so")


CALLS = calls_path()
CALLS_SOURCES = [os.path.join(HERE, "csrc", "paged_calls.cpp")]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def stale(target: str = LIB, sources=tuple(SOURCES + HEADERS)) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in [*sources, __file__])


def _start(cmd: list, target: str):
    """Starts cmd + ["-o", a temporary file], to become ``target``."""
    tmp = target + f".tmp{os.getpid()}"
    return subprocess.Popen(cmd + ["-o", tmp]), tmp, target


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec else ""


def calls_need() -> str:
    """What is missing here to build the extension module; empty: nothing."""
    torch_dir = _torch_dir()
    for what, there in (("g++", shutil.which("g++")), ("torch", torch_dir),
                        ("Python's headers", os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))),
                        ("torch's headers", os.path.exists(os.path.join(torch_dir, "include", "torch", "csrc", "autograd",
                                                                        "python_variable.h")))):
        if not there:
            return what
    return ""


def _start_calls():
    include, lib = (os.path.join(_torch_dir(), d) for d in ("include", "lib"))
    return _start(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
                   "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
                   "-isystem", sysconfig.get_paths()["include"]] + CALLS_SOURCES +
                  ["-L" + lib, "-lc10", "-ltorch_cpu", "-ltorch_python"], CALLS)


def build(force: bool = False, verbose: bool = False, calls: bool = True) -> str:
    """Builds what is missing or stale: the library, and (calls) the extension module, which
    is left out where there is no compiler, torch or header for it.  What has been built is
    in place even where the other one fails."""
    running = []
    if force or stale(LIB):
        cmd = [nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
               "-Xcompiler", "-fPIC", "-shared", "--threads", "0", "-I", os.path.join(ROOT, "include")] + SOURCES
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        running.append(_start(cmd, LIB))
    if calls and not calls_need() and (force or stale(CALLS, CALLS_SOURCES + HEADERS[:1])):
        running.append(_start_calls())
    failed = []
    for p, tmp, target in running:
        if p.wait():
            failed.append(p)
        else:
            os.replace(tmp, target)
    if failed:
        raise subprocess.CalledProcessError(failed[0].returncode, failed[0].args)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
