"""Build libtreeverify.so in-tree with nvcc for sm_100a, and the Python binding's marshalling
module (_marshal.so) with the host compiler against torch's headers."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libtreeverify.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo", "--threads", "0",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    # host arithmetic rounds each operation (the tree-shape DP compares sums exactly)
    "-Xcompiler", "-ffp-contract=off",
]


MARSHAL_SRC = os.path.join(PKG, "binding", "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_STAMP = os.path.join(PKG, "_marshal.built_for")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps += glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-shared", "-o", LIB, *sources()]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    return LIB


def marshal_target() -> str:
    """What a marshalling module is compiled for: another torch or Python needs another one."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def marshal_unavailable() -> str | None:
    """Why the marshalling module cannot be compiled here, or None."""
    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        return f"no C++ compiler ({cxx})"
    try:
        import torch
    except ImportError as e:
        return f"no torch ({e})"
    for d, name in ((os.path.join(os.path.dirname(torch.__file__), "include"), "ATen/core/Tensor.h"),
                    (sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(os.path.join(d, name)):
            return f"no {name} in {d}"
    return None


def build_marshal(force: bool = False, verbose: bool = False) -> str | None:
    """Needs libtreeverify.so (it is linked to it), a C++ compiler and the headers of torch and Python.  Where one of
    those is missing it says so and returns None: then everything but the wrappers of the cache calls works, and
    those raise."""
    why = marshal_unavailable()
    if why is not None:
        print(f"_marshal.so not built: {why}; decode_attention, evict_cache, rotary_write and cache_desc need it",
              file=sys.stderr)
        return None
    import torch
    deps = [MARSHAL_SRC, os.path.join(ROOT, "include", "treeverify.h")]
    target = marshal_target()
    built_for = None
    if os.path.exists(MARSHAL) and os.path.exists(MARSHAL_STAMP):
        with open(MARSHAL_STAMP) as f:
            built_for = f.read()
    if not force and built_for == target and all(os.path.getmtime(p) <= os.path.getmtime(MARSHAL) for p in deps):
        return MARSHAL
    base = os.path.dirname(torch.__file__)
    nvcc = shutil.which(os.environ.get("NVCC", "nvcc")) or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBUILT_FOR="{target}"',
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-o", MARSHAL, MARSHAL_SRC, "-L", PKG, "-l:libtreeverify.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    if os.path.exists(MARSHAL_STAMP):  # no module of an unfinished build passes for this one's
        os.remove(MARSHAL_STAMP)
    subprocess.check_call(cmd)
    with open(MARSHAL_STAMP, "w") as f:
        f.write(target)
    return MARSHAL


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    build_marshal(force="--force" in sys.argv, verbose=True)
