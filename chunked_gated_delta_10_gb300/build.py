"""Build the KDA CUDA library in-tree for sm_103a.

Compiles every ``csrc/*.cu`` file with nvcc (in parallel, one ``-gencode``)
and links ``lib/libkda_gb300.so``. No CMake, no torch extension machinery: the
library has a plain C ABI (``include/kda.h``, ``include/kda_serve.h``) and links
only the static CUDA runtime (TMA descriptors are encoded through the driver
entry point obtained at run time, so libcuda is not linked). Beside it
``lib/_kda_serve.so``: the Python module of the single-token operators, compiled
against PyTorch's headers (``csrc/serve_binding.cpp``). Where those or Python's are
not there (a PyTorch without CUDA, no ``Python.h``) it is left out, with a warning:
the library is built and the chunked operators run all the same.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

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


def _read(path):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _serve_missing():
    """What the Python module of the single-token operators cannot be compiled without and is not there, or None."""
    import torch

    if torch.version.cuda is None:
        return "a PyTorch with CUDA"
    for path in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                 os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "include", "ATen", "cuda", "EmptyTensor.h")):
        if not os.path.exists(path):
            return path
    return None


def _serve_commands(nvcc, obj):
    """Compile and link commands of the Python module of the single-token operators."""
    import torch

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


def _serve_made_by(commands):
    """What the module depends on besides its files: an object for another PyTorch or Python does not load, or worse."""
    import torch

    return "\n".join([torch.__version__, torch.__file__, sys.version, *(" ".join(c) for c in commands)])


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
    missing = _serve_missing()
    if missing:
        warnings.warn(f"{missing} is missing: {os.path.basename(SERVE)}, the Python module of the single-token operators, is "
                      "not built")
        if os.path.exists(SERVE):
            os.remove(SERVE)  # (another PyTorch's)
    else:
        compile_serve, link_serve = _serve_commands(nvcc, serve_obj)
        made_by, record = _serve_made_by([compile_serve, link_serve]), serve_obj + ".made_by"
        new = force or _stale(serve_obj, [SERVE_SRC] + headers) or _read(record) != made_by

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
        return r

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        serve = ex.submit(run, compile_serve) if not missing and new else None
        list(ex.map(run, jobs))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *objs, "-lcudart_static",
             "-lrt", "-ldl", "-lpthread"])
        os.replace(tmp, LIB)
    if serve:
        serve.result()  # (raises if it did not compile; the library is there by now)
    if not missing and (new or _stale(SERVE, [serve_obj, LIB])):
        tmp = SERVE + f".tmp{os.getpid()}"
        run([*link_serve, "-o", tmp])
        os.replace(tmp, SERVE)
        with open(record, "w") as f:
            f.write(made_by)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
