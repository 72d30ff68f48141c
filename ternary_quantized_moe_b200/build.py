"""Builds libscion.so in-tree with nvcc for sm_100a (B200).

Each .cu under csrc/ compiles to an object under _build/ (in parallel, skipped when
up to date), then everything links into ternary_quantized_moe_b200/libscion.so.
The CUDA runtime is linked statically, so the library loads on machines without a
GPU (every call then reports SCION_ECUDA).  csrc/binding.cpp, the CPython extension of
the per-token calls, compiles with the host compiler against torch's headers into
ternary_quantized_moe_b200/_binding.so.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libscion.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_KEY = os.path.join(BUILD, "binding.key")  # what the extension was built with
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src] + _deps()):
        cmd = [nvcc()] + ARCH + FLAGS + ["-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj + ".tmp"]
        subprocess.check_call(cmd)
        os.replace(obj + ".tmp", obj)
    return obj


def _binding_command(out: str) -> list:
    """The compiler's command for the extension: torch's headers, libraries and C++ ABI, this Python's headers."""
    import torch
    from torch.utils.cpp_extension import include_paths

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = include_paths() + [cuda, sysconfig.get_paths()["include"]]
    return ([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, '-DSCION_TORCH="%s"' % torch.__version__]
            + ["-isystem" + i for i in inc]
            + [os.path.join(CSRC, "binding.cpp"), "-o", out, "-L" + lib, "-Wl,-rpath," + lib,
               "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"])


def _binding_key() -> str:
    """What the extension depends on beside its sources (the command holds torch's version and paths)."""
    return "\n".join([sys.implementation.cache_tag] + _binding_command("_binding.so")) + "\n"


def _binding_stale() -> bool:
    if _stale(BINDING, [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "scion.h")]):
        return True
    if not os.path.exists(BINDING_KEY):
        return True
    with open(BINDING_KEY) as f:
        return f.read() != _binding_key()


def _build_binding() -> None:
    if not _binding_stale():
        return
    tmp = BINDING + ".tmp%d" % os.getpid()
    subprocess.check_call(_binding_command(tmp))
    os.replace(tmp, BINDING)
    with open(BINDING_KEY, "w") as f:
        f.write(_binding_key())


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with ThreadPoolExecutor(max_workers=min(9, len(sources) + 1)) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(_compile, sources))
        binding.result()
    if _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        subprocess.check_call([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"])
        os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
