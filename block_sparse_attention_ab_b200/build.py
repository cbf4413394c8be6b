"""Build libab_attn.so in-tree with nvcc for sm_100a (no JIT cache), and beside it _cache_bind.so,
the compiled Python binding of the key/value cache calls (host code only, torch's headers)."""

from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libab_attn.so")
SOURCES = ["ab_api.cu", "score_kernels.cu", "select_kernels.cu", "attn_kernel.cu", "ab_noalloc.cu",
           "ab_selftest.cu", "ab_host.cu", "attn_bwd_kernel.cu", "cache_api.cu", "cache_attn.cu",
           "cache_mass.cu", "cache_mass_tiles.cu",
           "cache_ops.cu", "cache_tiles.cu"]
HEADERS = ["ab_device.cuh", "ab_kernels.h", "cache_common.cuh", "cache_kernels.h",
           "cache_sched.cuh", "cache_tma.cuh", "tmap_host.h",
           os.path.join("..", "..", "include", "ab_attn.h")]
BINDING = os.path.join(HERE, "_cache_bind.so")
BINDING_SOURCE = "cache_bind.cpp"
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _stale(out, sources) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(p) > t for p in [os.path.join(CSRC, f) for f in sources] + [__file__])


def build_binding() -> str:
    """Compile _cache_bind.so against the running interpreter's torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    tmp = BINDING + ".tmp"
    subprocess.check_call(
        ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
         "-DTORCH_EXTENSION_NAME=_cache_bind", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
         *(f"-I{p}" for p in inc), os.path.join(CSRC, BINDING_SOURCE), "-o", tmp, f"-L{HERE}", "-l:libab_attn.so",
         f"-L{libs}", "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale(LIB, SOURCES + HEADERS):
        _build_library(verbose)
    if force or _stale(BINDING, [BINDING_SOURCE, HEADERS[-1]]):
        build_binding()
    return LIB


def _build_library(verbose: bool) -> str:
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs, jobs = [], []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [NVCC, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
               "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append((cmd, subprocess.Popen(cmd)))
        objs.append(obj)
    for cmd, job in jobs:
        if job.wait() != 0:
            raise subprocess.CalledProcessError(job.returncode, cmd)
    tmp = LIB + ".tmp"
    subprocess.check_call([NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
