"""Build ``libbitlinear.so`` (sm_100a) in the package directory with nvcc.

Each ``csrc/*.cu`` file is compiled to an object under ``_build/`` (in
parallel), then linked with the static CUDA runtime into one shared library
whose exported symbols are exactly the ``extern "C"`` functions of
``include/bitlinear.h``.  ``csrc/bl_calls.cpp`` (the Python side of the calls made
many times a step) is compiled with g++ against torch's headers into ``_calls.so``
beside it.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libbitlinear.so")
CALLS = os.path.join(HERE, "_calls.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    """Compile every CUDA source and link the library; returns its path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                     glob.glob(os.path.join(INCLUDE, "*.h")))
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_v:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_v:
            sys.stderr.write(r.stdout + r.stderr)

    with ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _build_calls(force)
    return LIB


def calls_stamp() -> str:
    """What _calls.so is compiled for: it holds this text, and loads into nothing else."""
    from importlib.metadata import version  # (importing torch takes seconds)
    return f"bl_calls for {sys.implementation.cache_tag}, torch {version('torch')}"


def calls_stale(path: str = CALLS) -> bool:
    """Whether _calls.so is missing, older than its sources, or of another Python or torch."""
    if _stale(path, [os.path.join(CSRC, "bl_calls.cpp"), os.path.join(INCLUDE, "bitlinear.h")]):
        return True
    with open(path, "rb") as f:
        return calls_stamp().encode() + b"\0" not in f.read()


def _build_calls(force: bool = False) -> None:
    """Compile csrc/bl_calls.cpp into _calls.so."""
    if not force and not calls_stale():
        return
    src = os.path.join(CSRC, "bl_calls.cpp")
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    incs = [*include_paths(), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBL_CALLS_STAMP="{calls_stamp()}"',
           "-I", INCLUDE,
           *(x for i in incs for x in ("-isystem", i)), src, "-o", tmp, "-L", libs, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-L", HERE, "-l:libbitlinear.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_v="--ptxas-v" in sys.argv)
    print(LIB)
