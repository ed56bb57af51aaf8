"""Builds the KDA CUDA library (libkda.so) in-tree for sm_103a.

Each .cu file in csrc/ is compiled as its own translation unit (in parallel)
with ``-gencode arch=compute_103a,code=sm_103a -lineinfo``, then linked into
``_build/libkda.so``.  No cmake, no torch extension machinery: the library is a
plain C-ABI shared object loaded with ctypes.  Beside it, csrc/cache_binding.cpp becomes
an extension module of this Python and torch, by the host compiler in one step.  Where that fails (no headers
of Python, a compiler that torch's do not take) the library is built all the same, with a warning: the recurrent
layer's calls need no more, and the global-attention operators raise when they are used.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libkda.so")
BINDING_SRC = os.path.join(CSRC, "cache_binding.cpp")
BINDING = os.path.join(OUT_DIR, f"kda_cache_binding-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")

CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return (sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(CSRC, "*.h")))
            + sorted(glob.glob(os.path.join(INCLUDE, "*.h"))))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src] + _headers()):
        cmd = [NVCC] + ARCH + FLAGS + ["-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stderr)
    return obj


def _compile_binding(force: bool) -> str:
    """Builds the binding; returns what went wrong, if anything did.  None of other sources is left then."""
    if force or _stale(BINDING, [BINDING_SRC] + _headers()):
        tmp = BINDING + f".tmp{os.getpid()}"
        root = os.path.dirname(torch.__file__)
        includes = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                    sysconfig.get_path("include"), os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
        cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
        for d in includes:
            cmd += ["-isystem" if d is not INCLUDE else "-I", d]
        cmd += [BINDING_SRC, "-o", tmp, "-L" + os.path.join(root, "lib")]
        cmd += ["-l" + name for name in ("c10", "c10_cuda", "torch_cpu", "torch", "torch_python")]
        try:
            r = subprocess.run(cmd, capture_output=True, text=True)
            failed = f"{r.stdout}\n{r.stderr}" if r.returncode != 0 else ""
        except OSError as e:
            failed = str(e)
        if failed:
            if os.path.exists(BINDING):
                os.remove(BINDING)
            return f"{CXX} failed for {BINDING_SRC}:\n{failed}"
        os.replace(tmp, BINDING)
    return ""


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles every csrc/*.cu for sm_103a and links libkda.so, and builds the binding, of whose failure it only
    warns; returns the library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = _sources()
    if force:
        for o in glob.glob(os.path.join(OUT_DIR, "*.o")):
            os.remove(o)
    with ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding, force)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if binding.result():
        warnings.warn(f"the global-attention operators' binding was not built: {binding.result()}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
