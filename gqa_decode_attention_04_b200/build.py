"""Build the CUDA library in-tree: csrc/*.cu (+ host-only csrc/*.cpp) -> libgqa_decode.so
(sm_100a only), and the binding's marshalling module csrc/fastcall.cc -> _fastcall.<key>.so.

Usage:  python -m gqa_decode_attention_04_b200.build [--verbose]
The shared object is written next to this file so it travels with the source tree.
"""
from __future__ import annotations

import glob
import hashlib
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgqa_decode.so")
FAST_SOURCE = os.path.join(CSRC, "fastcall.cc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-v",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def needs_rebuild() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def fastcall_path() -> str:
    """Where the marshalling module for this Python, this torch and these sources is.  The name says what it was
    built for, so one that was built for others is never loaded, and is not there when asked for."""
    import torch
    key = hashlib.sha256(repr((sys.version_info[:3], sysconfig.get_config_var("SOABI"), torch.__version__)).encode())
    for path in [FAST_SOURCE, *sorted(glob.glob(os.path.join(INCLUDE, "*.h")))]:
        with open(path, "rb") as f:
            key.update(f.read())
    return os.path.join(HERE, f"_fastcall.{key.hexdigest()[:16]}.so")


def build_fastcall(verbose: bool = False, force: bool = False) -> str:
    """The extension module that checks and passes torch tensors (host code only)."""
    fast = fastcall_path()
    if not force and os.path.exists(fast):
        return fast
    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    tmp = fast + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-shared", "-fPIC", "-std=c++17",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"], FAST_SOURCE, "-o", tmp,
           "-L", lib, "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {FAST_SOURCE}")
    for old in glob.glob(os.path.join(HERE, "_fastcall*.so")):
        os.remove(old)
    os.replace(tmp, fast)
    return fast


def build(verbose: bool = False, force: bool = False) -> str:
    """The library, then the marshalling module, which it does not need: without a C++ compiler or the headers of
    Python or torch the calls go through ctypes."""
    build_library(verbose, force)
    try:
        build_fastcall(verbose, force)
    except (RuntimeError, OSError) as e:
        sys.stderr.write(f"{e}: built without the marshalling module\n")
    return LIB


def build_library(verbose: bool = False, force: bool = False) -> str:
    if not force and not needs_rebuild():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True)
    print(LIB)
