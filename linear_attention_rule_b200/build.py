"""Build in-tree: libkda.so for sm_100a with nvcc (no JIT cache, no torch in it), and, where torch is
installed, kda_native.so, the binding's argument marshalling for the calls of a decode step, with the
host compiler against torch."""
from __future__ import annotations

import importlib.util
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkda.so")
NATIVE_SRC = os.path.join(PKG, "native", "kda_native.cpp")
NATIVE = os.path.join(PKG, "kda_native.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))] + [
        os.path.join(INCLUDE, "libkda.h")]


def _stale(target: str, inputs) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(s) > os.path.getmtime(target) for s in inputs)


def needs_build() -> bool:
    return _stale(LIB, sources())


def _run(cmd, target: str, verbose: bool) -> None:
    """Run a compiler that writes to a file of its own, then put that in the target's place."""
    tmp = target + ".tmp.%d" % os.getpid()
    cmd = cmd + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, target)


def torch_version():
    """The installed torch's version, without importing it; None where there is no torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    with open(os.path.join(spec.submodule_search_locations[0], "version.py")) as fh:
        return re.search(r"^__version__ = ['\"](.*?)['\"]", fh.read(), re.M).group(1)


def native_needs_build() -> bool:
    """Older than its sources, or built against another torch (whose version it holds)."""
    if _stale(NATIVE, [NATIVE_SRC, os.path.join(INCLUDE, "libkda.h")]):
        return True
    with open(NATIVE, "rb") as fh:
        return b"kda_native for torch " + torch_version().encode() + b"\0" not in fh.read()


def build_native(force: bool = False, verbose: bool = False) -> str:
    if not force and not native_needs_build():
        return NATIVE
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")))
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include")] + cpp_extension.include_paths()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
    cmd += ['-DKDA_TORCH_VERSION="%s"' % torch_version()]
    cmd += [x for d in includes for x in ("-isystem", d)] + [NATIVE_SRC]
    cmd += [x for d in cpp_extension.library_paths() for x in ("-L" + d, "-Wl,-rpath," + d)]
    _run(cmd + ["-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], NATIVE, verbose)
    return NATIVE


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if force or needs_build():
        nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
        _run([nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + [
            "-I", INCLUDE, "-I", CSRC, os.path.join(CSRC, "libkda.cu")], LIB, verbose)
    if torch_version() is None:
        print("no torch: kda_native.so, which only the Python binding needs, is not built", file=sys.stderr)
    else:
        build_native(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv)
    print(LIB)
