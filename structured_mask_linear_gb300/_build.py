"""Builds the C-ABI shared library libloglinear.so in-tree with nvcc for sm_103a, and the
CPython module _native.so (csrc/binding.cpp) against the installed torch with g++.

Each translation unit compiles in parallel to an object file under _build/, then one
nvcc link makes _build/libloglinear.so (CUDA runtime linked statically).  Rebuilds
only when a source or header is newer than the library, the module also when torch has
changed.  Without the interpreter's headers the module is left out, with a warning.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libloglinear.so")
BINDING = os.path.join(CSRC, "binding.cpp")
NATIVE = os.path.join(OUT_DIR, "_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libloglinear.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _torch_version() -> str:
    import torch

    return torch.__version__


def native_up_to_date() -> bool:
    stamp = NATIVE + ".torch"
    if not (os.path.exists(NATIVE) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        if f.read() != _torch_version():
            return False
    t = os.path.getmtime(NATIVE)
    return all(os.path.getmtime(p) <= t for p in [BINDING] + glob.glob(os.path.join(INCLUDE, "*.h")))


def _native_command(out: str):
    import torch
    from torch.utils import cpp_extension

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if cxx is None:
        raise RuntimeError("g++ not found: it is required to build _native.so")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    paths = [sysconfig.get_paths()["include"], INCLUDE, os.path.join(cuda, "include")] + cpp_extension.include_paths()
    return ([cxx, "-shared", "-fPIC", "-O2", "-std=c++17", BINDING, "-o", out] + [f"-I{p}" for p in paths] +
            [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-L{lib}", f"-Wl,-rpath,{lib}",
             "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"])


def native_missing() -> str:
    """What the CPython module cannot be built without and is not there; empty if nothing is."""
    header = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    return "" if os.path.exists(header) else f"{header} (the interpreter's headers)"


def build(force: bool = False, verbose: bool = False) -> str:
    native, missing = None, native_missing()
    if missing:  # the library does not need the module; the calls that do raise
        warnings.warn(f"_native.so is not built: {missing} is missing", RuntimeWarning, stacklevel=2)
    elif force or not native_up_to_date():
        os.makedirs(OUT_DIR, exist_ok=True)
        tmp = NATIVE + f".tmp{os.getpid()}"
        cmd = _native_command(tmp)
        native = (tmp, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
    try:
        _build_library(force, verbose)
    finally:
        if native is not None:
            tmp, cmd, p = native
            out, _ = p.communicate()
    if native is not None:
        if p.returncode != 0:
            raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + out.decode(errors="replace"))
        os.replace(tmp, NATIVE)
        with open(NATIVE + ".torch", "w") as f:
            f.write(_torch_version())
    return LIB


def _build_library(force: bool, verbose: bool) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-I", INCLUDE, "--expt-relaxed-constexpr"]
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc, "-c", src, "-o", obj] + common
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((src, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, cmd, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append(f"{' '.join(cmd)}\n{text}")
        elif verbose and text:
            print(text)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, "-shared", "-o", tmp] + objs + ARCH, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
