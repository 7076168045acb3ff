"""Builds libimc.so (the CUDA library behind include/imc.h) in-tree for sm_103a.

Each translation unit is compiled in parallel with nvcc, then linked into a
shared library next to this file; beside it the Python module over its 4-bit and
expert entry points (_calls), for the Python that runs the build, where that has
its headers.  Rebuilds only when a source or header is newer than the library.
Usage: ``python -m addmm_implicit_im2col_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libimc.so")
CALLS_PATH = os.path.join(HERE, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
CALLS_SOURCE = os.path.join(CSRC, "calls.c")
SOURCES = ["imc_api.cu", "k_simt.cu", "k_tc_gemm.cu", "k_tc_conv.cu", "noalloc.cu", "mx_api.cu",
           "k_mx_quant.cu", "k_mx_gemm.cu", "k_experts.cu", "k_balance.cu", "k_adapters.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def common_flags():
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
            "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES] + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def is_stale(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in _inputs())


def is_calls_stale() -> bool:
    if not os.path.exists(CALLS_PATH):
        return True
    t = os.path.getmtime(CALLS_PATH)
    return any(os.path.getmtime(p) > t for p in (CALLS_SOURCE, os.path.join(INCLUDE, "imc.h")))


def _compile(src: str, verbose: bool, ptxas_info: bool):
    obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
    cmd = [nvcc(), *common_flags(), "-c", src, "-o", obj]
    if ptxas_info:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _link_calls():
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        # libimc.so is whole without it, and the binding calls through ctypes instead
        print(f"no Python.h in {include}: _calls is not built", file=sys.stderr)
        return
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CC", "gcc"), "-O2", "-shared", "-fPIC", "-I", INCLUDE,
           "-I", include, CALLS_SOURCE, "-o", tmp, "-L", HERE,
           "-l:" + os.path.basename(LIB_PATH), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building _calls failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compiles and links libimc.so; returns its path."""
    if force or is_stale():
        os.makedirs(BUILD_DIR, exist_ok=True)
        srcs = [os.path.join(CSRC, s) for s in SOURCES]
        with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
            objs = list(ex.map(lambda s: _compile(s, verbose, ptxas_info), srcs))
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
    if force or is_calls_stale():
        _link_calls()
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv))
