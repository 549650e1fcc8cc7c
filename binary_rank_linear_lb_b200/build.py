"""Build liblb.so (the C-ABI CUDA library) in-tree for sm_100a.

    python -m binary_rank_linear_lb_b200.build [--verbose]

Compiles every ``csrc/*.cu`` with nvcc for ``sm_100a`` only and links them into
``binary_rank_linear_lb_b200/liblb.so``, and ``csrc/lb_torch.cpp`` (the dense path's argument
marshalling for torch tensors) with g++ into ``lb_torch.so`` beside it.  Runs without a GPU
(nvcc cross-compiles).  Where g++, torch or Python's headers are missing, liblb.so is built
alone, with a warning: its C ABI needs none of them.  (Without torch the package cannot be
imported; run this file by its path.)
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "liblb.so")
EXT = os.path.join(PKG, "lb_torch.so")
STAMP = os.path.join(PKG, "_build", "lb_torch.made_for")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                              glob.glob(os.path.join(CSRC, "*.h"))) + [
        os.path.join(ROOT, "include", "lb.h")]


def ext_deps():
    return [os.path.join(CSRC, "lb_torch.cpp"), os.path.join(ROOT, "include", "lb.h")]


def newer(target, sources_) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in sources_)


def made_for() -> str:
    """What lb_torch.so fits: the installed torch and this Python (neither shows in the times
    of its sources)."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "none"
    return f"torch {torch} {sysconfig.get_config_var('SOABI')}\n"


def ext_current() -> bool:
    if not newer(EXT, ext_deps()) or not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == made_for()


def up_to_date() -> bool:
    return newer(LIB, deps()) and ext_current()


def ext_lacks() -> Optional[str]:
    """What is missing to build lb_torch.so, or None."""
    if shutil.which("g++") is None:
        return "no g++"
    if importlib.util.find_spec("torch") is None:
        return "no torch"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "no Python headers"
    return None


def build_ext() -> None:
    """lb_torch.so, and beside the objects what it was made for."""
    if os.path.exists(STAMP):
        os.remove(STAMP)
    compile_ext()
    os.makedirs(os.path.dirname(STAMP), exist_ok=True)
    with open(STAMP, "w") as f:
        f.write(made_for())


def compile_ext() -> None:
    """lb_torch.so, linked against the liblb.so beside it and the installed torch."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    tmp = EXT + f".tmp{os.getpid()}"
    subprocess.check_call([
        "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + os.path.join(ROOT, "include"),
        "-I" + os.path.join(base, "include"),
        "-I" + os.path.join(base, "include", "torch", "csrc", "api", "include"),
        "-I" + os.path.join(cuda, "include"), "-I" + sysconfig.get_paths()["include"],
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        os.path.join(CSRC, "lb_torch.cpp"), "-o", tmp, "-L" + os.path.join(base, "lib"), "-lc10",
        "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python", "-L" + PKG,
        "-l:liblb.so", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, EXT)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    if force or not newer(LIB, deps()):
        build_lib(verbose)
    lacks = ext_lacks()
    if lacks is None:
        build_ext()
    else:
        if os.path.exists(EXT) and not ext_current():      # of other sources: better none
            os.remove(EXT)
        warnings.warn(f"lb_torch.so is not built ({lacks}): liblb.so is complete, the dense "
                      "path's Python functions will raise")
    return LIB


def build_lib(verbose: bool = False) -> None:
    out_dir = os.path.join(PKG, "_build")
    os.makedirs(out_dir, exist_ok=True)
    nvcc = nvcc_path()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I" + os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    objs = []
    for src in sources():
        obj = os.path.join(out_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcuda", "-lcublas",
                           "-lcusolver"])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
