"""In-tree build of libattn_gb300.so for sm_103a.

Every ``csrc/*.cu`` file is compiled by nvcc in parallel into ``_build/`` and
linked into ``libattn_gb300.so`` next to this file; ``csrc/native.cpp``, the compiled
part of the Python binding, becomes ``_native.so`` beside it (host code only, with
PyTorch's headers).  The CUDA runtime is linked
statically and the driver is reached through the runtime's entry-point query,
so the library also loads (for symbol checks) on a machine without a GPU
driver.  Objects are rebuilt only when a source or header is newer.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libattn_gb300.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
INCLUDE_DIR = os.path.join(os.path.dirname(PKG_DIR), "include")
NATIVE_SRC = os.path.join(CSRC, "native.cpp")
NATIVE_PATH = os.path.join(PKG_DIR, "_native.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "-Xptxas", "-warn-spills", f"-I{INCLUDE_DIR}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn_gb300.so")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(INCLUDE_DIR, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(nvcc: str, src: str, obj: str, verbose: bool):
    cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        sys.stderr.write(res.stdout + res.stderr)
    return obj


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _compile_native(nvcc: str, verbose: bool):
    import torch
    root = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    includes = [INCLUDE_DIR, os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = NATIVE_PATH + ".tmp"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in includes],
           NATIVE_SRC, "-o", tmp, f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu",
           "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding did not compile:\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, NATIVE_PATH)


def build(verbose: bool = False, jobs: int | None = None) -> str:
    """Compile (as needed) and link the library; return its path."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    todo = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if _stale(obj, [src, *headers]):
            todo.append((src, obj))
    # rebuilt for another PyTorch too
    native = _stale(NATIVE_PATH, [NATIVE_SRC, os.path.join(INCLUDE_DIR, "attn_gb300.h"),
                                  os.path.join(_torch_dir(), "version.py")])
    if todo or native:
        workers = jobs or min(len(todo) + native, os.cpu_count() or 4)
        with cf.ThreadPoolExecutor(max_workers=workers) as ex:
            jobs_ = [ex.submit(_compile_native, nvcc, verbose)] if native else []
            jobs_ += [ex.submit(_compile, nvcc, src, obj, verbose) for src, obj in todo]
            for job in jobs_:
                job.result()
    if todo or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp"
        cmd = [nvcc, *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
