"""Builds the CUDA library (libgdn.so, sm_103a) in-tree with nvcc.

Each .cu file under csrc/ is compiled to an object in parallel, then linked
into ``_lib/libgdn.so``; csrc/attn_bind.cpp becomes the Python extension module
``_lib/_attn_bind.so`` beside it (against the running interpreter and torch).
Nothing is installed outside the package directory.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libgdn.so")
BIND_SRC = os.path.join(CSRC, "attn_bind.cpp")
BIND_PATH = os.path.join(LIB_DIR, "_attn_bind.so")
BIND_FOR = os.path.join(LIB_DIR, "_attn_bind.for")   # the interpreter and torch that it was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps()) and _bind_up_to_date()


def _bind_for() -> str:
    import torch
    return "%s %s %s" % (sysconfig.get_config_var("SOABI"), torch.__version__, torch.__file__)


def _bind_up_to_date() -> bool:
    if not os.path.exists(BIND_PATH) or not os.path.exists(BIND_FOR):
        return False
    t = os.path.getmtime(BIND_PATH)
    with open(BIND_FOR) as f:
        same = f.read() == _bind_for()
    return same and all(os.path.getmtime(p) <= t for p in
                        (BIND_SRC, os.path.join(INCLUDE, "gdn.h"), os.path.abspath(__file__)))


def _compile_bind() -> str:
    """The object of the extension module (host code only)."""
    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    obj = os.path.join(BUILD_DIR, "attn_bind.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()), "-I", INCLUDE, "-I", root, "-I",
           os.path.join(root, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"], "-I", cuda,
           "-c", BIND_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on %s:\n%s\n%s" % (BIND_SRC, " ".join(cmd), r.stdout + r.stderr))
    return obj


def _link_bind(obj: str) -> None:
    import torch
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND_PATH + ".%d.tmp" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", LIB_DIR, "-lgdn", "-L", torch_lib, "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stdout + r.stderr))
    os.replace(tmp, BIND_PATH)
    with open(BIND_FOR, "w") as f:
        f.write(_bind_for())


def build_library(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, " ".join(cmd), r.stdout + r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        bind = ex.submit(_compile_bind)
        objs = list(ex.map(compile_one, srcs))
        bind_obj = bind.result()
    tmp = LIB_PATH + ".%d.tmp" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stdout + r.stderr))
    os.replace(tmp, LIB_PATH)
    _link_bind(bind_obj)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose=True))
