"""Build the sm_103a shared library in-tree (``_build/librmsnorm_gb300.so``).

Each kernel translation unit is compiled by its own nvcc process in parallel,
then linked with the C-ABI unit into one shared library that exports only
the ``rmsnorm_*`` symbols of ``include/rmsnorm.h``.  The CUDA runtime is
linked statically, so the library needs nothing but the driver at run time.
The attention-path operators (``csrc_attn``) are built the same way into a
library of their own (``_build/librmsnorm_attn_gb300.so``, the ``rmsattn_*``
symbols of ``include/rmsnorm_attn.h``).  Both need nvcc alone.  The module that
marshals the attention path's Python calls is compiled against torch and
Python; without torch there is nothing to marshal and it is left out.

``build(checked=True)`` makes the bounds-checked debug library
(``_build/librmsnorm_gb300_checked.so``, compiled with -DRMSNORM_BOUNDS_CHECK):
every global access and ring copy of its kernels is checked against its
tensor's extent, and one out of range is skipped and reported in bit 1 of the
status word.  Point the binding at it with the environment variable
RMSNORM_GB300_LIB.
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
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "librmsnorm_gb300.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
CHECKED_PATH = os.path.join(BUILD_DIR, "librmsnorm_gb300_checked.so")
# the attention-path operators, a library of their own
ATTN_CSRC = os.path.join(PKG, "csrc_attn")
ATTN_PATH = os.path.join(BUILD_DIR, "librmsnorm_attn_gb300.so")
# native marshalling of its tensor-level calls (a Python extension module)
FAST_SRC = os.path.join(PKG, "binding", "attn_fast.cpp")


def fast_path() -> str:
    """The module's file for this torch, Python and machine: it is compiled
    against their object layouts, so another one's is not loaded."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "unknown"
    return os.path.join(BUILD_DIR, f"rmsattn_fast-torch{torch}-{sysconfig.get_config_var('SOABI')}.so")


FAST_PATH = fast_path()
# the bench's C timing harness (not part of the library)
HOSTCOST_SRC = os.path.join(PKG, "bench_src", "host_cost.cu")
HOSTCOST_PATH = os.path.join(BUILD_DIR, "librmsn_hostcost.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler",
              "-fvisibility=hidden", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def attn_sources() -> list[str]:
    return sorted(glob.glob(os.path.join(ATTN_CSRC, "*.cu")))


def _inputs(checked: bool = False) -> list[str]:
    """What the libraries are made of; ``checked``: the row norm's alone."""
    dirs = [CSRC] if checked else [CSRC, ATTN_CSRC]
    return ([f for d in dirs for ext in ("cu", "cuh", "h", "inc") for f in glob.glob(os.path.join(d, "*." + ext))]
            + ([os.path.join(INCLUDE, "rmsnorm.h")] if checked else glob.glob(os.path.join(INCLUDE, "*.h")))
            + [os.path.abspath(__file__)] + ([] if checked else [HOSTCOST_SRC, FAST_SRC]))


def _torch_dir() -> str | None:
    """Where torch is installed, if it is."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _fast_command(torch_dir: str, out: str) -> list[str]:
    """g++ of the marshalling module: torch's and Python's headers, host code
    only; torch's own libraries are loaded before it."""
    inc = os.path.join(torch_dir, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
            "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda,
            "-I", sysconfig.get_paths()["include"], FAST_SRC, "-o", out,
            "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def up_to_date(checked: bool = False) -> bool:
    outs = [CHECKED_PATH] if checked else [LIB_PATH, ATTN_PATH, HOSTCOST_PATH]
    if not checked and _torch_dir():
        outs.append(FAST_PATH)
    if not all(os.path.exists(o) for o in outs):
        return False
    t = min(os.path.getmtime(o) for o in outs)
    return all(os.path.getmtime(f) <= t for f in _inputs(checked))


def build(force: bool = False, verbose: bool = False, jobs: int | None = None,
          checked: bool = False) -> str:
    """Compile and link the libraries (the bounds-checked row-norm one with
    ``checked``) if a source is newer; return the row-norm library's path."""
    out = CHECKED_PATH if checked else LIB_PATH
    if not force and up_to_date(checked):
        return out
    obj_dir = os.path.join(BUILD_DIR, "checked") if checked else BUILD_DIR
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()
    srcs = sources() + ([] if checked else attn_sources())
    objs = [os.path.join(obj_dir, os.path.basename(s)[:-3] + ".o") for s in srcs]
    extra = ["-DRMSNORM_BOUNDS_CHECK"] if checked else []

    def compile_one(pair):
        src, obj = pair
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    def compile_fast(torch_dir):
        # the C ABI's symbols stay undefined: that library is loaded before it
        tmp = FAST_PATH + f".tmp{os.getpid()}"
        r = subprocess.run(_fast_command(torch_dir, tmp), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {os.path.basename(FAST_SRC)}:\n{r.stderr}")
        os.replace(tmp, FAST_PATH)

    n = jobs or min(len(srcs), os.cpu_count() or 1)
    with ThreadPoolExecutor(max(1, n)) as ex:
        torch_dir = None if checked else _torch_dir()
        fast = ex.submit(compile_fast, torch_dir) if torch_dir else None
        logs = list(ex.map(compile_one, zip(srcs, objs)))
    if verbose:
        for src, log in zip(srcs, logs):
            sys.stderr.write(f"== {os.path.basename(src)}\n{log}")
    n_norm = len(sources())
    for lib, part in [(out, objs[:n_norm])] + ([] if checked else [(ATTN_PATH, objs[n_norm:])]):
        tmp = lib + f".tmp{os.getpid()}"
        link = [cc, *ARCH, "-shared", "-cudart", "static", *part, "-o", tmp]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if checked:
        return out
    # the C timing harness, linked against the library it times
    tmp = HOSTCOST_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, *NVCC_FLAGS, "-shared", "-cudart", "static", HOSTCOST_SRC, "-o", tmp,
           "-L", BUILD_DIR, "-lrmsnorm_gb300", "-Xlinker", "-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host-cost harness failed to build:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, HOSTCOST_PATH)
    if fast is not None:
        fast.result()  # raises if it failed: the C libraries are there all the same
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                checked="--checked" in sys.argv))
