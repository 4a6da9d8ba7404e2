"""Builds libneattn.so (the CUDA library behind include/ne_attn.h) in-tree.

nvcc compiles each translation unit for sm_103a in parallel, then links a
shared library with the CUDA runtime linked statically (the driver API is
reached through cudaGetDriverEntryPointByVersion, so libcuda is not linked).
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libneattn.so")
BIND_SOURCE = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(BUILD, "_neattn_bind.so")  # the compiled part of binding.py, for this interpreter and torch
SOURCES = ["api.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_decode.cu", "qkv_proj.cu", "qk_norm.cu", "paged.cu",
           "paged_prefix.cu", "paged_plan.cu", "paged_tree.cu"]
HEADERS = ["ptx.cuh", "rope.cuh", "internal.h", "paged.cuh", "paged_sweep.cuh", "paged_prefix.cuh"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _newest_input():
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    paths.append(os.path.join(HERE, "..", "include", "ne_attn.h"))
    paths += [os.path.abspath(__file__), BIND_SOURCE]
    return max(os.path.getmtime(p) for p in paths)


def _compile_bind():
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    lib = os.path.join(root, "lib")
    tmp = BIND + ".%d.tmp" % os.getpid()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-I" + p for p in inc]
           + [BIND_SOURCE, "-o", tmp, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for bind.cpp:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, BIND)


def build(force=False, verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    newest = _newest_input()
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= newest for p in (LIB, BIND)):
        return LIB
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [NVCC] + ARCH + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(_compile_bind)
        objs = list(ex.map(compile_one, SOURCES))
        bind.result()
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
