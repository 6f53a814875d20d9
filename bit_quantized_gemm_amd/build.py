"""Build libatom.so (the C-ABI library) for gfx950 with hipcc, and the Python extension module ``_short`` (the binding's
short way into it) with the host compiler, in-tree.

Usage: ``python -m bit_quantized_gemm_amd.build``.  Objects go to ``_build/``; the shared
libraries are written next to this file.  Every call recompiles.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libatom.so")
SHORT = os.path.join(HERE, "_short" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["atom_api.cpp", "select.hip", "quantize.hip", "gemm.hip", "gemm_small.hip", "gemm_w4a8.hip",
           "serve_api.cpp", "w8a8_quantize.hip", "gemm_w8a8.hip", "kv4_cache.hip", "kv4_attention.hip",
           "mxfp4_api.cpp", "mxfp4_quantize.hip", "gemm_mxfp4.hip", "rmsnorm.hip", "kv4_pages_api.cpp", "kv4_pages.hip"]

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17",
    # never emit packed fp32 arithmetic (v_pk_{add,mul,fma}_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # IEEE fp32 division and denormals: the scale rounding rule depends on them
    "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-gpu-flush-denormals-to-zero",
    "-fno-fast-math", "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC, *COMMON, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


class Unavailable(RuntimeError):
    """Something that the extension module is built with is not there (the C library needs none of it)."""


def _build_short() -> None:
    """The extension module, against the headers and libraries of the torch that will load it."""
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError as e:
        raise Unavailable(f"torch is not importable ({e})") from None
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx or not shutil.which(cxx):
        raise Unavailable("there is no host C++ compiler (g++, or CXX)")
    python = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(python, "Python.h")):
        raise Unavailable(f"Python's headers are not installed ({python})")
    from . import _built_for

    include = [*cpp_extension.include_paths(), python]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [cxx, "-O2", "-fPIC", "-std=c++17", "-Wall", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DATOM_BUILT_FOR="{_built_for()}"', f"-I{INCLUDE}", *(a for i in include for a in ("-isystem", i)), os.path.join(CSRC, "short_calls.cpp"), "-o", SHORT + ".tmp",
           f"-L{lib}", "-lc10", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for short_calls.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(SHORT + ".tmp", SHORT)
    untagged = os.path.join(os.path.dirname(SHORT), "_short.so")      # of builds that named no Python
    if untagged != SHORT and os.path.exists(untagged):
        os.remove(untagged)


def build(verbose: bool = False) -> str:
    """Both libraries.  The C library needs hipcc alone: it is linked first, and where the extension module cannot be built for want of
    torch, a host compiler or Python's headers, that is said on stderr and an older one removed (the binding works without)."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        short = ex.submit(_build_short)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    built = [LIB]
    try:
        short.result()
        built.append(SHORT)
    except Unavailable as e:
        if os.path.exists(SHORT):
            os.remove(SHORT)
        print(f"{os.path.basename(SHORT)} is not built: {e}; calls take the binding's full checks", file=sys.stderr)
    if verbose:
        print("built " + " and ".join(built))
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
