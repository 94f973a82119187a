"""Build libpae.so (the C-ABI library of include/pae.h) in-tree for sm_100a, and
_int8_tensors.so, the tensor side of int8.py, against the installed PyTorch.

    python -m flow_matching_action_pi0_b200.build [--force] [--verbose]

nvcc cross-compiles for sm_100a without a GPU.  The static CUDA runtime is
linked in and the driver's tensor-map encoder is fetched at run time, so the
library loads on a machine without a GPU (only the calls need one).
"""
from __future__ import annotations

import argparse
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libpae.so")
TENSORS = os.path.join(HERE, "_int8_tensors.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


_TENSORS_SRC = os.path.join(CSRC, "int8_tensors.cpp")


def _tensors_command():
    import torch
    from torch.utils import cpp_extension as ext
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no C++ compiler found")
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
            *(f"-isystem{p}" for p in (*ext.include_paths("cuda"), sysconfig.get_paths()["include"])),
            _TENSORS_SRC, "-o", TENSORS + ".tmp", *(f"-L{p}" for p in ext.library_paths("cuda")),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _newer(target: str, deps) -> bool:
    """`target` is there and no file of `deps` is newer."""
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps)


def _torch_version():
    """The installed PyTorch, None without one (looked up without importing it)."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def _lib_current() -> bool:
    return _newer(LIB, sources() + [p for pat in ("*.cuh", "*.h") for p in glob.glob(os.path.join(CSRC, pat))] +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _tensors_current() -> bool:
    stamp = _stamp()
    if not _newer(TENSORS, [_TENSORS_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == _torch_version()


def _stamp() -> str:
    """The file that says which PyTorch the tensor module was built against."""
    return os.path.join(HERE, "_build", os.path.basename(TENSORS) + ".torch")


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    """libpae.so first, which needs nvcc alone, then the tensor module where
    PyTorch is installed; a tensor module that does not compile is an error, but
    leaves libpae.so in place."""
    os.makedirs(os.path.join(HERE, "_build"), exist_ok=True)
    if force or not _lib_current():
        _build_lib(verbose, ptxas_v)
    version = _torch_version()
    if version is None:
        print(f"PyTorch is not installed: {os.path.basename(TENSORS)} is left out, int8.py needs it")
    elif force or not _tensors_current():
        _build_tensors(version, verbose)
    return LIB


def _build_tensors(version: str, verbose: bool) -> None:
    cmd = _tensors_command()
    if verbose:
        print(" ".join(cmd))
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if p.returncode:
        sys.stdout.write(p.stdout)
        raise RuntimeError(f"compilation failed for: {_TENSORS_SRC} ({LIB} is built)")
    os.replace(TENSORS + ".tmp", TENSORS)
    with open(_stamp(), "w") as f:
        f.write(version)


def _build_lib(verbose: bool, ptxas_v: bool) -> None:
    objdir = os.path.join(HERE, "_build")
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                    "-I", INCLUDE, "-I", CSRC]
    if ptxas_v:
        flags += ["-Xptxas", "-v"]
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc()] + flags + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or ptxas_v or p.returncode):
            sys.stdout.write(out)
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs + ["-lcudart_static", "-ldl",
                                                                                      "-lpthread", "-lrt"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force or a.ptxas_v, verbose=a.verbose, ptxas_v=a.ptxas_v))
