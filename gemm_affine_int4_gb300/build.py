"""Build libgai4.so in-tree: every csrc/*.cu compiled for sm_103a in parallel
with nvcc, then linked into one shared library next to this file (the CUDA
runtime is linked statically, so the library loads on hosts without a GPU
driver too), and _calls.so, the module that reaches some of its entries from
Python without ctypes (csrc/torch_calls.cpp, g++ against PyTorch's headers; left
out where there is no PyTorch for CUDA: the library needs none).
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


def _torch():
    """(folder, text of its version file) of a PyTorch for CUDA, or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    folder = os.path.dirname(spec.origin)
    if not glob.glob(os.path.join(folder, "lib", "libtorch_cuda.so*")):
        return None
    with open(os.path.join(folder, "version.py")) as f:
        return folder, f.read()


def _calls_command(nvcc: str, torch: str, obj: str):
    """(compile, link) of torch_calls.cpp; the module finds libgai4.so beside itself."""
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
               sysconfig.get_paths()["include"]]
    compile_ = ["g++", "-std=c++17", "-O2", "-Wall", "-fPIC", "-c", os.path.join(CSRC, "torch_calls.cpp"), "-o", obj]
    for d in include:
        compile_ += ["-isystem", d]
    link = ["g++", "-shared", obj, "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L" + HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def _calls_key(version: str, commands) -> str:
    """What _calls.so is made for, beside its sources: layouts of PyTorch's and Python's objects."""
    return "\n".join([version, sys.version, str(sysconfig.get_config_var("EXT_SUFFIX"))] + [" ".join(c) for c in commands])


def _made_for(stamp: str, key: str) -> bool:
    if not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == key


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

    torch = _torch()
    calls_src = os.path.join(CSRC, "torch_calls.cpp")
    calls_obj, stamp = os.path.join(BUILD, "torch_calls.o"), os.path.join(BUILD, "torch_calls.key")
    if torch is None:
        print("no PyTorch for CUDA: libgai4.so is built without _calls.so, which calls some of its entries from Python",
              file=sys.stderr)
    else:
        commands = _calls_command(nvcc, torch[0], calls_obj)
        key = _calls_key(torch[1], commands)
        if force or _stale(calls_obj, [calls_src] + deps) or not _made_for(stamp, key):
            if os.path.exists(stamp):
                os.remove(stamp)
            jobs.insert(0, (calls_src, commands[0]))

    def run(job):
        src, cmd = job
        p = subprocess.run(cmd, capture_output=True, text=True)
        return src, p.returncode, p.stdout + p.stderr

    failed = []
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for src, rc, log in ex.map(run, jobs):
                if verbose or rc != 0:
                    sys.stderr.write(log)
                if rc != 0:
                    failed.append(src)

    def link(target, cmd):
        tmp = target + ".tmp%d" % os.getpid()
        p = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
        if p.returncode != 0:
            sys.stderr.write(p.stdout + p.stderr)
            raise RuntimeError(f"linking {os.path.basename(target)} failed")
        os.replace(tmp, target)

    # (the library first: it does not need the module)
    if not set(failed) - {calls_src} and (force or jobs or _stale(LIB, objs)):
        link(LIB, [nvcc] + ARCH + ["-shared"] + objs)
    if failed:
        raise RuntimeError("compiling " + ", ".join(os.path.basename(f) for f in failed) + " failed")
    if torch is not None and (force or jobs or _stale(CALLS, [calls_obj]) or not _made_for(stamp, key)):
        link(CALLS, commands[1])
        with open(stamp, "w") as f:
            f.write(key)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
