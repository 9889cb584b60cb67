"""Build libsvdq.so (the CUDA library behind include/svdq.h) for sm_100a, and
_bind.*.so (the argument marshalling of its tensor operators).

``build()`` compiles the library, which needs nvcc alone; ``build_bind()`` the
marshalling, which needs the installed torch and a C++ compiler (the first call
of a tensor operator runs it).  ``python -m
bit_diffusion_transformer_w4a4_b200.build`` does both, the second where torch is
installed.  The shared objects are written next to this file so that they
travel with the source tree; they are rebuilt when any source is newer.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsvdq.so")
OBJ = os.path.join(HERE, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "svdq.h")])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, file=sys.stderr)


def bind_path() -> str:
    """The marshalling module of this interpreter and the installed torch: it
    uses torch's C++ interface, which changes from build to build, so each has
    a file of its own."""
    import torch
    tag = f"{sys.implementation.cache_tag}-torch{torch.__version__}-{(torch.version.git_version or '')[:8]}"
    return os.path.join(HERE, f"_bind.{re.sub('[^0-9A-Za-z.-]', '_', tag)}.so")


def bind_stale() -> bool:
    path = bind_path()
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in (os.path.join(CSRC, "bind.cpp"), os.path.join(ROOT, "include", "svdq.h")))


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """Compile the marshalling against the installed torch (its libraries are
    loaded by ``import torch``, which comes first)."""
    path = bind_path()
    if not force and not bind_stale():
        return path
    import torch
    from torch.utils.cpp_extension import include_paths
    inc = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(ROOT, "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = f"{path}.{os.getpid()}.tmp"
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[f"-I{i}" for i in inc], os.path.join(CSRC, "bind.cpp"), "-o", tmp,
          "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], verbose)
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """The library; returns its path."""
    if not force and not stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objs = [os.path.join(OBJ, os.path.basename(u) + ".o") for u in units]
    inc = ["-I", os.path.join(ROOT, "include")]
    with concurrent.futures.ThreadPoolExecutor() as ex:
        list(ex.map(lambda uo: _run([nvcc(), *NVCC_FLAGS, *(extra or []), *inc, "-c", uo[0], "-o", uo[1]], verbose),
                    zip(units, objs)))
    _run([nvcc(), *LINK_FLAGS, *objs, "-o", LIB + ".tmp"], verbose)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
    print(LIB)
    if importlib.util.find_spec("torch"):
        print(build_bind(force="--force" in sys.argv, verbose=True))
