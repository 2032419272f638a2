"""Build libgai4.so in-tree: every csrc/*.cu compiled for sm_103a in parallel
with nvcc, then linked into one shared library next to this file (the CUDA
runtime is linked statically, so the library loads on hosts without a GPU
driver too), and _calls.so, the module that reaches some of its entries from
Python without ctypes (csrc/torch_calls.cpp, g++ against PyTorch's headers).
Usage: python -m gemm_affine_int4_gb300.build [--verbose]."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(os.path.dirname(HERE), "_build")
LIB = os.path.join(HERE, "libgai4.so")
CALLS = os.path.join(HERE, "_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                     "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgai4.so")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  [os.path.join(os.path.dirname(HERE), "include", "gai4.h")])


def _calls_command(nvcc: str, obj: str):
    """(compile, link) of torch_calls.cpp; the module finds libgai4.so beside itself."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
               sysconfig.get_paths()["include"]]
    compile_ = ["g++", "-std=c++17", "-O2", "-Wall", "-fPIC", "-c", os.path.join(CSRC, "torch_calls.cpp"), "-o", obj]
    for d in include:
        compile_ += ["-isystem", d]
    link = ["g++", "-shared", obj, "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L" + HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def build(verbose: bool = False, force: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    deps = _deps()
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + deps):
            cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
            jobs.append((src, cmd))

    calls_obj = os.path.join(BUILD, "torch_calls.o")
    compile_calls, link_calls = _calls_command(nvcc, calls_obj)
    calls_src = compile_calls[compile_calls.index("-c") + 1]
    if force or _stale(calls_obj, [calls_src] + deps):
        jobs.insert(0, (calls_src, compile_calls))

    def run(job):
        src, cmd = job
        p = subprocess.run(cmd, capture_output=True, text=True)
        return src, p.returncode, p.stdout + p.stderr

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
            for src, rc, log in ex.map(run, jobs):
                if verbose or rc != 0:
                    sys.stderr.write(log)
                if rc != 0:
                    raise RuntimeError(f"compiling {os.path.basename(src)} failed")

    def link(target, cmd):
        tmp = target + ".tmp%d" % os.getpid()
        p = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
        if p.returncode != 0:
            sys.stderr.write(p.stdout + p.stderr)
            raise RuntimeError(f"linking {os.path.basename(target)} failed")
        os.replace(tmp, target)

    if force or jobs or _stale(LIB, objs):
        link(LIB, [nvcc] + ARCH + ["-shared"] + objs)
    if force or jobs or _stale(CALLS, [calls_obj]):
        link(CALLS, link_calls)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
