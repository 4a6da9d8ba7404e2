"""Builds libneattn.so (the CUDA library behind include/ne_attn.h) in-tree.

nvcc compiles each translation unit for sm_103a in parallel, then links a
shared library with the CUDA runtime linked statically (the driver API is
reached through cudaGetDriverEntryPointByVersion, so libcuda is not linked).
g++ compiles the part of binding.py that is C++ against the installed torch.
"""
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libneattn.so")
HEADER = os.path.join(HERE, "..", "include", "ne_attn.h")
BIND_SOURCE = "bind.cpp"  # the compiled part of binding.py
SOURCES = ["api.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_decode.cu", "qkv_proj.cu", "qk_norm.cu", "paged.cu",
           "paged_prefix.cu", "paged_plan.cu", "paged_tree.cu"]
HEADERS = ["ptx.cuh", "rope.cuh", "internal.h", "paged.cuh", "paged_sweep.cuh", "paged_prefix.cuh"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _stale(path, sources):
    """Whether `path` is missing or older than one of its inputs."""
    inputs = [os.path.join(CSRC, f) for f in sources] + [HEADER, os.path.abspath(__file__)]
    return not os.path.exists(path) or os.path.getmtime(path) < max(os.path.getmtime(p) for p in inputs)


def bind_path():
    """The compiled part of binding.py.  It uses the interpreter's and torch's C++ interfaces, so its name says which."""
    import torch
    return os.path.join(BUILD, "_neattn_bind.torch-%s%s" % (torch.__version__, sysconfig.get_config_var("EXT_SUFFIX")))


def _build_bind(force):
    try:
        path = bind_path()
    except ModuleNotFoundError as e:
        if e.name != "torch":
            raise
        sys.stderr.write("torch is not installed: the compiled part of its binding is left out\n")
        return
    if not force and not _stale(path, [BIND_SOURCE]):
        return
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    lib = os.path.join(root, "lib")
    tmp = path + ".%d.tmp" % os.getpid()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-I" + p for p in inc]
           + [os.path.join(CSRC, BIND_SOURCE), "-o", tmp, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (BIND_SOURCE, r.stdout, r.stderr))
    os.replace(tmp, path)


def _build_lib(ex, verbose):
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

    objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)


def build(force=False, verbose=False):
    """Builds what is out of date and returns the library's path.  The library needs no torch; the compiled part of the
    binding does: it is left out where torch is not installed, and where it does not compile this raises once the library
    is there."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(_build_bind, force)
        if force or _stale(LIB, SOURCES + HEADERS):
            _build_lib(ex, verbose)
        bind.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
