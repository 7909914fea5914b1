"""Build libssd.so (CUDA for sm_100a, with nvcc) and the native Python binding
_bind.so (with g++, against torch's headers) in-tree.

Each ``csrc/*.cu`` file is compiled separately (in parallel) into ``_build/``
and linked into ``selective_state_space_22_b200/libssd.so``.  The CUDA runtime
is linked statically and the driver library is not linked at all (the tensor
map encoder is fetched through the runtime's entry-point query), so the
library also loads on a host without a GPU driver.

    python -m selective_state_space_22_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libssd.so")
BIND = os.path.join(PKG, "_bind.so")
BIND_FOR = os.path.join(BUILD, "_bind.for")  # the Python and torch that BIND was built against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libssd.so")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_for() -> str:
    from importlib.metadata import version

    return f"{sys.version}\ntorch {version('torch')}\n"


def _bind_stale() -> bool:
    """Whether the binding is older than its sources or was built against another Python or torch."""
    if _stale(BIND, [os.path.join(CSRC, "bind.cpp"), os.path.join(INCLUDE, "ssd.h"), __file__]):
        return True
    try:
        with open(BIND_FOR) as f:
            return f.read() != _bind_for()
    except OSError:
        return True


def _bind_command() -> list[str]:
    import sysconfig

    import torch

    t = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [INCLUDE, os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(t, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-I{i}" for i in inc], os.path.join(CSRC, "bind.cpp"), "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python", f"-Wl,-rpath,{lib}"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every kernel source for sm_100a, link libssd.so and the binding; return the library's path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    hdrs = _headers()
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s, __file__] + hdrs):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)
    bind_tmp = None
    if force or _bind_stale():
        bind_tmp = BIND + f".tmp{os.getpid()}"
        jobs.append([*_bind_command(), "-o", bind_tmp])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        for out in ex.map(run, jobs):
            if verbose and out:
                print(out)
    if bind_tmp:
        os.replace(bind_tmp, BIND)
        with open(BIND_FOR, "w") as f:
            f.write(_bind_for())
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
