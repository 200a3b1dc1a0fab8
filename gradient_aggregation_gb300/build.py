"""Builds the engine's CUDA library in-tree: ``_build/libfc.so``.

Every ``csrc/*.cu`` file is compiled for sm_103a in parallel with nvcc and
linked into one shared library with the CUDA runtime linked statically (the
library then needs only the driver at run time).  No CMake, no setuptools.

``csrc/fc_bind.cpp``, the tensor checks of the training-step operators' Python
binding, becomes a Python module for the torch that is installed
(``build_binding``).  The library needs neither it nor torch, g++'s Python headers
or Python: ``build_library`` builds it alone, ``build_all`` both side by side.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libfc.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
BIND_SRC = os.path.join(CSRC, "fc_bind.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return (sorted(glob.glob(os.path.join(CSRC, "*.cuh")))
            + sorted(glob.glob(os.path.join(CSRC, "*.h")))
            + [os.path.join(INCLUDE, "fc.h")])


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def bind_path() -> str:
    """Where the Python module is: one for each Python and torch, it is of no use to
    another."""
    import torch
    return os.path.join(OUT_DIR, "_fcbind.%s.torch-%s.so" % (
        sys.implementation.cache_tag, torch.__version__.replace("+", "-")))


def _bind_command(target: str):
    """The compiler call that makes the Python module."""
    import torch
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("a C++ compiler is required to build the Python binding")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    home = os.path.dirname(torch.__file__)
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(home, "include"),
           os.path.join(home, "include", "torch", "csrc", "api", "include"), cuda]
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
            *["-I" + d for d in inc], BIND_SRC, "-o", target,
            "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
            "-lc10"]


def build_binding(force: bool = False) -> str:
    """Compile (if needed) the Python module for the installed torch and return its
    path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    path = bind_path()
    if force or _stale(path, [BIND_SRC, os.path.join(INCLUDE, "fc.h"), __file__]):
        part = path + ".tmp.%d" % os.getpid()
        p = subprocess.run(_bind_command(part), stdout=subprocess.PIPE,
                           stderr=subprocess.STDOUT, text=True)
        if p.returncode != 0:
            sys.stderr.write(p.stdout)
            raise RuntimeError("building the Python binding failed")
        os.replace(part, path)
    return path


def build_all(force: bool = False, verbose: bool = False) -> str:
    """The library and the Python module, side by side; returns the path of libfc.so.
    If the module cannot be built, the library is there all the same."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        bind = ex.submit(build_binding, force)
        path = build_library(force, verbose)
        bind.result()
    return path


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libfc.so."""
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = _sources()
    hdrs = _headers()
    if not force and not _stale(LIB_PATH, srcs + hdrs + [__file__]):
        return LIB_PATH
    nvcc = _nvcc()
    objs = []
    jobs = []
    for src in srcs:
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC,
               "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append(cmd)

    def run(cmd):
        p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                           text=True)
        return cmd, p.returncode, p.stdout

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(run, jobs))
    for cmd, rc, out in results:
        if verbose or rc != 0:
            sys.stderr.write(out)
        if rc != 0:
            raise RuntimeError("nvcc failed: " + " ".join(cmd))
    tmp = LIB_PATH + ".tmp.%d" % os.getpid()
    link = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-ldl"]
    p = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if p.returncode != 0:
        sys.stderr.write(p.stdout)
        raise RuntimeError("link failed: " + " ".join(link))
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    make = build_library if "--library" in sys.argv else build_all
    print(make(force="--force" in sys.argv, verbose="-v" in sys.argv))
