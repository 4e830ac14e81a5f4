"""Build the sm_100a shared library ``libunipin.so`` (nvcc) and the Python calls into it (calls_module(), g++,
against the installed torch), in-tree."""

from __future__ import annotations

import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libunipin.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
    "--expt-relaxed-constexpr",
    "-shared", "--threads", "4",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) \
        + [os.path.join(INCLUDE, "unipin.h")]


def calls_module() -> str:
    """Name of the compiled module of the paged and windowed calls.  It is built against one torch, whose version
    is part of the name (and Python's ABI of the file's): under another one it is a module yet to be built."""
    import torch
    return "_calls_torch_" + re.sub(r"\W", "_", torch.__version__)


def calls_path() -> str:
    import sysconfig
    return os.path.join(PKG, calls_module() + sysconfig.get_config_var("EXT_SUFFIX"))


def _calls_deps():
    return [os.path.join(CSRC, "calls.cpp"), os.path.join(INCLUDE, "unipin.h")]


def _newer(target, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and _newer(calls_path(), _calls_deps())


def _build_calls(verbose: bool):
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    target = calls_path()
    tmp = target + ".tmp.%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-DCALLS_MODULE=" + calls_module()]
    for d in (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE):
        cmd += ["-I", d]
    cmd += ["-o", tmp, os.path.join(CSRC, "calls.cpp"), "-L", PKG, "-l:libunipin.so", "-L", os.path.join(root, "lib"),
            "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    """Compile every .cu under csrc/ into libunipin.so (static cudart, no libcuda link) and calls.cpp into
    the module calls_module()."""
    if not force and up_to_date():
        return LIB
    if force or not _newer(LIB, _deps()):
        nvcc = os.environ.get("NVCC", "nvcc")
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [nvcc] + NVCC_FLAGS + list(extra or []) + ["-I", INCLUDE, "-I", CSRC, "-o", tmp] + _sources()
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    if force or not _newer(calls_path(), _calls_deps()):
        _build_calls(verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
