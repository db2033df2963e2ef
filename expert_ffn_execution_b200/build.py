"""Builds libstrata_moe.so in-tree with nvcc for sm_100a.

Each .cu under csrc/ is compiled to an object (in parallel) and linked into one
shared library next to this file; native/mxcalls.cpp becomes the Python module
_mxcalls beside it (g++, the CPython and torch headers), where it can be built:
without it the same calls run in Python.  Run `python -m expert_ffn_execution_b200.build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libstrata_moe.so")
CALLS_SRC = os.path.join(HERE, "native", "mxcalls.cpp")
# named for this interpreter: another's neither finds it nor takes it for its own
CALLS = os.path.join(HERE, "_mxcalls" + sysconfig.get_config_var("EXT_SUFFIX"))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + [os.path.join(INCLUDE, "strata_moe.h")])


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_calls(force: bool = False) -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    torch_dir = os.path.dirname(spec.origin)
    deps = (CALLS_SRC, os.path.join(INCLUDE, "strata_moe.h"), os.path.join(torch_dir, "version.py"))
    if not force and os.path.exists(CALLS) and all(
            os.path.getmtime(p) <= os.path.getmtime(CALLS) for p in deps):
        return CALLS
    import torch  # its headers and libraries, which are loaded before the module is
    at = os.path.join(torch_dir, "include")
    libs = ("c10", "c10_cuda", "torch_cpu", "torch_cuda", "torch_python")
    cuda = os.path.dirname(os.path.dirname(NVCC))
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-Wall", "-shared", "-fPIC",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DSTRATA_TORCH="{torch.__version__}"', "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
           "-isystem", at, "-isystem", os.path.join(at, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), CALLS_SRC, "-o", CALLS + ".tmp",
           "-L", os.path.join(torch_dir, "lib"), *("-l" + n for n in libs)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALLS_SRC}:\n{r.stderr}")
    os.replace(CALLS + ".tmp", CALLS)
    return CALLS


def try_build_calls(force: bool = False) -> str | None:
    """The native module or, where it cannot be built (no compiler, no Python
    headers, a torch without CUDA or with other headers), None and a warning."""
    # an older build's name, which any interpreter would import
    for old in {os.path.join(HERE, "_mxcalls.so")} - {CALLS}:
        if os.path.exists(old):
            os.remove(old)
    try:
        return build_calls(force)
    except Exception as e:  # whatever is missing: the module is optional
        if os.path.exists(CALLS):
            os.remove(CALLS)  # of other sources or another torch
        warnings.warn(f"_mxcalls was not built, the microscaled calls run in Python: {e}")
        return None


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    lib = build_library(force, verbose_ptxas)
    try_build_calls(force)
    return lib


def build_library(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), _sources()))
    tmp = LIB + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
