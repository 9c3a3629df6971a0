"""Build libmoefp8.so in-tree with nvcc for sm_100a (B200).

    python -m mixture_experts_fp8_b200.build [--force] [--verbose]

Each .cu under csrc/ is compiled to an object under _build/ (in parallel, skipped when up to
date) and linked with the static CUDA runtime into mixture_experts_fp8_b200/libmoefp8.so.
`--debug` (or build_all()) also builds libmoefp8_debug.so from the same sources with
MOE_FAULT_INJECTION, the library the failure-detection tests inject faults through.  The
driver API entry point used for TMA descriptors is fetched at run time, so the library does not
link libcuda.

csrc/binding.cpp, the Python module that marshals the operators around the layer, is compiled by the
host compiler against PyTorch's headers into mixture_experts_fp8_b200/_binding.so.  Where PyTorch is not
installed the libraries alone are built.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoefp8.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "binding.for")   # the PyTorch and Python that it was built for
# The debug library: the same sources with MOE_FAULT_INJECTION, for failure-detection tests.
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libmoefp8_debug.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoefp8.so")
    return exe


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, verbose: bool, build_dir: str = BUILD, defines=()) -> str:
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *[f"-D{d}" for d in defines], "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Build libmoefp8.so (or, with debug=True, libmoefp8_debug.so) and return its path."""
    build_dir, lib = (BUILD_DEBUG, LIB_DEBUG) if debug else (BUILD, LIB)
    defines = ("MOE_FAULT_INJECTION",) if debug else ()
    os.makedirs(build_dir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    dep = _deps_mtime()
    todo = []
    for s in srcs:
        obj = os.path.join(build_dir, os.path.basename(s) + ".o")
        if force or verbose or not os.path.exists(obj) or os.path.getmtime(obj) < max(dep, os.path.getmtime(s)):
            todo.append(s)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        list(ex.map(lambda s: _compile(s, verbose, build_dir, defines), todo))
    objs = [os.path.join(build_dir, os.path.basename(s) + ".o") for s in srcs]
    if todo or not os.path.exists(lib) or os.path.getmtime(lib) < max(os.path.getmtime(o) for o in objs):
        tmp = lib + f".{os.getpid()}.tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
        os.replace(tmp, lib)
    return lib


def binding_matches() -> bool:
    """Whether _binding.so is there and was built for this PyTorch and Python (its C++ interface differs by release)."""
    try:
        with open(BINDING_FOR) as f:
            return os.path.exists(BINDING) and f.read() == _binding_for()
    except OSError:
        return False


def _binding_for() -> str:
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}\n"


def build_binding(force: bool = False) -> str:
    """Build _binding.so (host code only) and return its path."""
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src, os.path.join(INCLUDE, "moefp8.h")]
    if not force and binding_matches() and os.path.getmtime(BINDING) >= max(map(os.path.getmtime, deps)):
        return BINDING
    import torch
    os.makedirs(BUILD, exist_ok=True)
    base = os.path.dirname(torch.__file__)
    includes = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = BINDING + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           *[f for p in includes for f in ("-isystem", p)], src, "-o", tmp, "-L", os.path.join(base, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {src}:\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        f.write(_binding_for())
    os.replace(tmp, BINDING_FOR)
    return BINDING


def _bindings(force: bool) -> list:
    return [build_binding(force)] if importlib.util.find_spec("torch") else []


def build_all(force: bool = False, verbose: bool = False) -> list:
    """The release library, the fault-injection debug library and (where PyTorch is) the Python module."""
    return [build(force, verbose), build(force, False, debug=True), *_bindings(force)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/spill usage")
    ap.add_argument("--debug", action="store_true", help="also build libmoefp8_debug.so")
    a = ap.parse_args()
    print(build_all(a.force, a.verbose) if a.debug else
          [build(force=a.force, verbose=a.verbose), *_bindings(a.force)])
