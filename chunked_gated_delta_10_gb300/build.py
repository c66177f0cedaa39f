"""Build the KDA CUDA library in-tree for sm_103a.

Compiles every ``csrc/*.cu`` file with nvcc (in parallel, one ``-gencode``)
and links ``lib/libkda_gb300.so``. No CMake, no torch extension machinery: the
library has a plain C ABI (``include/kda.h``, ``include/kda_serve.h``) and links
only the static CUDA runtime (TMA descriptors are encoded through the driver
entry point obtained at run time, so libcuda is not linked). Beside it
``lib/_kda_serve.so``: the Python module of the single-token operators, compiled
against PyTorch's headers (``csrc/serve_binding.cpp``).
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIB_DIR, "libkda_gb300.so")
SERVE = os.path.join(LIB_DIR, "_kda_serve.so")
SERVE_SRC = os.path.join(CSRC, "serve_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I" + os.path.join(ROOT, "include")]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the KDA CUDA library cannot be built")
    return exe


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _serve_commands(nvcc, obj):
    """Compile and link commands of the Python module of the single-token operators."""
    top = os.path.dirname(os.path.abspath(torch.__file__))
    include = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
               sysconfig.get_paths()["include"]]
    cxx = shutil.which("g++") or "g++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                *[x for d in include for x in ("-isystem", d)], "-c", SERVE_SRC, "-o", obj]
    link = [cxx, "-shared", obj, LIB, "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(top, "lib"), "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"]
    return compile_, link


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if stale) and return the path of the shared library."""
    nvcc = _nvcc()
    os.makedirs(OBJ, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    headers = _headers()
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
            jobs.append(cmd)
    serve_obj = os.path.join(OBJ, "serve_binding.o")
    compile_serve, link_serve = _serve_commands(nvcc, serve_obj)
    if force or _stale(serve_obj, [SERVE_SRC] + headers):
        jobs.insert(0, compile_serve)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
        return r

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        list(ex.map(run, jobs))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *objs, "-lcudart_static",
             "-lrt", "-ldl", "-lpthread"])
        os.replace(tmp, LIB)
    if force or _stale(SERVE, [serve_obj, LIB]):
        tmp = SERVE + f".tmp{os.getpid()}"
        run([*link_serve, "-o", tmp])
        os.replace(tmp, SERVE)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
