"""Builds the sm_100a shared library ``libvit_b200.so`` in-tree with nvcc.

``python -m resolution_vit_vision_b200.build`` (or ``build()``) compiles every ``csrc/*.cu`` and
``csrc/*.cpp`` for ``-gencode arch=compute_100a,code=sm_100a`` and links them, with the CUDA
runtime linked statically, into ``resolution_vit_vision_b200/libvit_b200.so``; then
``csrc/binding/vit_call.cpp`` with the host compiler, against the installed torch and that library, into
the extension module ``_vit_call.so`` beside it. Objects are cached under
``resolution_vit_vision_b200/_build`` and rebuilt when a source or header is newer.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libvit_b200.so")
CALL_SRC = os.path.join(CSRC, "binding", "vit_call.cpp")
CALL = os.path.join(PKG, "_vit_call.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest and not verbose_ptxas:
        return obj
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd = [nvcc()] + NVCC_FLAGS + ["-x", "cu"] + ARCH + ["-c", src, "-o", obj]
    if verbose_ptxas and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}\n{r.stdout}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _compile_call() -> str:
    """The extension module's object: host code only, so torch's headers meet the host compiler alone."""
    import sysconfig

    import torch
    obj = os.path.join(BUILD, "vit_call.o")
    newest = max(os.path.getmtime(f) for f in [CALL_SRC, torch.version.__file__] + glob.glob(os.path.join(ROOT, "include", "*.h")))
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wno-attributes",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-isystem", sysconfig.get_paths()["include"], "-c", CALL_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {CALL_SRC} failed:\n{r.stderr}\n{r.stdout}")
    return obj


def _link_call(obj: str) -> None:
    import torch
    if os.path.exists(CALL) and os.path.getmtime(CALL) >= max(os.path.getmtime(obj), os.path.getmtime(LIB)):
        return
    tmp = CALL + ".tmp"
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libvit_b200.so", "-Wl,-rpath,$ORIGIN",
           f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {CALL} failed:\n{r.stderr}\n{r.stdout}")
    os.replace(tmp, CALL)


def build(verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        call = ex.submit(_compile_call)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        tmp = LIB + ".tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}\n{r.stdout}")
        os.replace(tmp, LIB)
    _link_call(call.result())
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv))
