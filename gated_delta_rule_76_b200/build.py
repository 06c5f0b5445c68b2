"""Build libgdn.so (CUDA for sm_100a) in-tree with nvcc.

Every .cu file under csrc/ is compiled to an object in parallel, then linked into
gated_delta_rule_76_b200/libgdn.so.  Usage: ``python -m gated_delta_rule_76_b200.build``.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
SELFTEST_LIB = os.path.join(PKG, "libgdn_selftest.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def selftest_sources():
    return sorted(glob.glob(os.path.join(CSRC, "selftest", "*.cu")))


def _deps(srcs):
    return srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date(lib, srcs) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps(srcs))


def binding() -> str:
    """Path of the binding's native module for this torch and this Python, whose ABI it takes."""
    import torch
    return os.path.join(PKG, f"_attn_calls-torch{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build(force: bool = False, verbose: bool = False, jobs: int = 0) -> str:
    """Build libgdn.so, the binding's native module (where the host can) and the test-only libgdn_selftest.so; returns the libgdn.so path."""
    _build_lib(SELFTEST_LIB, selftest_sources(), "selftest_", force, verbose, jobs)
    _build_lib(LIB, sources(), "", force, verbose, jobs)
    _build_binding(force, verbose)
    _look_again()
    return LIB


def _look_again():
    """A binding that was looked for before it was built is looked for again at the next call."""
    gdn = sys.modules.get(f"{__package__}.gdn")
    if gdn is not None and gdn.__dict__.get("_native", gdn) is None:
        del gdn._native


def _build_binding(force, verbose):
    """The native marshalling of the attention layer's short calls, against torch's headers.  Every call does without it
    (more slowly), so that a host on which it does not build is told, and keeps the library."""
    src = os.path.join(CSRC, "binding", "attn_calls.cpp")
    path = binding()
    if not force and up_to_date(path, [src]):
        return
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    tmp = path + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", src, "-o", tmp, "-I", INCLUDE, "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-I", sysconfig.get_paths()["include"], "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = "" if r.returncode == 0 else r.stdout + r.stderr
    except OSError as e:
        why = str(e)
    if why:
        if os.path.exists(path):
            os.remove(path)  # of older sources
        warnings.warn(f"the binding's native module is not built, calls are marshalled through ctypes: g++ on "
                      f"{os.path.basename(src)}: {why}")
        return
    os.replace(tmp, path)


def _build_lib(lib, srcs, prefix, force, verbose, jobs):
    if not force and up_to_date(lib, srcs):
        return lib
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, prefix + os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=jobs or max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
