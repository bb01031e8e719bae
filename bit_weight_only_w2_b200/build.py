"""Build liblowbit.so (the CUDA library) in-tree with nvcc for sm_100a.

    python -m bit_weight_only_w2_b200.build [--force] [--debug]

Objects go to ``_build/`` at the repository root; the shared library is written next to this
file so the Python binding (and a copy of the tree on another machine) finds it, and beside it
_marshal.so, which marshals the arguments of the binding's short calls (g++ and PyTorch's headers;
where they are missing the library is built all the same). ``--debug``
builds liblowbit_debug.so instead: the same sources with device-side index checks
(LOWBIT_DEBUG_CHECKS), objects in ``_build/debug/``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "liblowbit.so")
DEBUG_LIB = os.path.join(PKG, "liblowbit_debug.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL_LIB = os.path.join(PKG, "_marshal.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I" + INCLUDE, "-I" + CSRC]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hdrs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hdrs


def _stale(target, inputs):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def _compile(src, obj, verbose, extra=()):
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    out_dir = os.path.join(BUILD, "debug") if debug else BUILD
    lib = DEBUG_LIB if debug else LIB
    extra = ("-DLOWBIT_DEBUG_CHECKS",) if debug else ()
    os.makedirs(out_dir, exist_ok=True)
    deps = _deps()
    objs = []
    jobs = []
    for src in sources():
        obj = os.path.join(out_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, *deps]):
            jobs.append((src, obj))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
            for log in ex.map(lambda j: _compile(j[0], j[1], verbose, extra), jobs):
                if verbose and log:
                    sys.stderr.write(log)
    if force or jobs or _stale(lib, objs):
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fvisibility=hidden"]
        subprocess.check_call(cmd)
        os.replace(tmp, lib)
    if not debug:
        build_marshal(force)
    return lib


def build_marshal(force: bool = False) -> Optional[str]:
    """Build _marshal.so against the installed PyTorch; the binding uses it with that version only, and does
    without it where it is missing. So where it cannot be built (no PyTorch, no C++ compiler, no headers) this
    says so on stderr and returns None."""
    try:
        return _build_marshal(force)
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(MARSHAL_LIB):   # (of other sources or another PyTorch)
            os.remove(MARSHAL_LIB)
        print(f"_marshal.so was not built, the binding marshals in Python: {e}", file=sys.stderr)
        return None


def _build_marshal(force: bool) -> str:
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    if not force and not _stale(MARSHAL_LIB, [MARSHAL_SRC, os.path.join(INCLUDE, "lowbit.h"), torch.version.__file__]):
        return MARSHAL_LIB
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(NVCC))
    headers = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = MARSHAL_LIB + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DLOWBIT_TORCH_VERSION="{torch.__version__.split("+")[0]}"', f"-I{INCLUDE}",
           *(f"-isystem{h}" for h in headers), MARSHAL_SRC,
           "-o", tmp, f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL_LIB)
    return MARSHAL_LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
