"""Build the native library libpkv.so (CUDA kernels for sm_103a + host allocator)
and the extension _bind-*.so, the Python entry of its shortest calls.

Usage: python -m paged_kv_cache_276_gb300.build [--force]

Translation units are compiled in parallel with nvcc, then linked into
``paged_kv_cache_276_gb300/_build/libpkv.so`` (in-tree, git-ignored).  The CUDA
runtime is linked statically, so the library only needs the driver at run time.
The extension beside it is compiled against Python's and a CUDA PyTorch's C++
headers, which the library does not need: where they are missing the library is
built all the same, with a warning, and the calls that go through the extension
raise.  Its file name carries the PyTorch and Python that it was built for
(native.bind_path), so another one's is never loaded.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libpkv.so")

SOURCES = ["decode.cu", "chunk_tc.cu", "cache_ops.cu", "quant_ops.cu", "decode_quant.cu", "rope_ops.cu", "spans.cu",
           "spans_tc.cu", "spans_step.cu", "alloc.cpp", "step.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "pkv.h"))
    files.append(os.path.abspath(__file__))
    return files


def _fresh(path: str) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in _deps())


def _bind_path() -> str:
    """The extension's file; its name takes PyTorch, which the library builds without."""
    if ROOT not in sys.path:
        sys.path.append(ROOT)
    from paged_kv_cache_276_gb300 import native
    return native.bind_path()


def _bind_fresh() -> bool:
    try:
        return _fresh(_bind_path())
    except ImportError:
        return False


def up_to_date() -> bool:
    return _fresh(LIB) and _bind_fresh()


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    cmd = [nvcc(), "-c", path, "-o", obj, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC] + ARCH
    if src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"] if os.environ.get("PKV_PTXAS_VERBOSE") else []
    else:
        cmd += ["-x", "c++"]
    subprocess.run(cmd, check=True)
    return obj


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _compile_bind() -> str:
    obj = os.path.join(BUILD, "bind.o")
    torch_inc = os.path.join(_torch_dir(), "include")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    subprocess.run(["g++", "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj, "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE,
                    "-I", sysconfig.get_paths()["include"], "-I", torch_inc,
                    "-I", os.path.join(torch_inc, "torch", "csrc", "api", "include"), "-I", cuda_inc], check=True)
    return obj


def _link_bind(obj: str):
    path = _bind_path()
    tmp = path + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", obj, "-o", tmp, "-L", BUILD, "-l:libpkv.so", "-Wl,-rpath,$ORIGIN",
                    "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"],
                   check=True)
    os.replace(tmp, path)


_bind_failed = False  # not tried again in this process


def build(force: bool = False) -> str:
    """Build what is missing or older than its sources; returns the library's path.  The library comes
    first: an extension that cannot be built costs a warning, not the library."""
    global _bind_failed
    lib_due = force or not _fresh(LIB)
    bind_due = force or lib_due or not (_bind_failed or _bind_fresh())
    if not lib_due and not bind_due:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(_compile_bind) if bind_due else None
        objs = list(ex.map(_compile, SOURCES)) if lib_due else []
    if lib_due:
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static"], check=True)
        os.replace(tmp, LIB)
    if bind_due:
        try:
            _link_bind(bind.result())
            _bind_failed = False
        except (ImportError, OSError, RuntimeError, subprocess.CalledProcessError) as e:
            _bind_failed = True
            warnings.warn(f"{LIB} is built, but not its Python extension, which the 8-bit cache's calls need: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv))
