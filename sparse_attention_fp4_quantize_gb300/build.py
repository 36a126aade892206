"""Build libcsa2.so in-tree: every .cu in csrc/ compiled for sm_103a (in
parallel), then linked into one shared library next to this file; and beside
it _csa2_bind.so, the Python extension (csrc/bind.cpp)."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libcsa2.so")
BIND = os.path.join(HERE, "_csa2_bind.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch() -> str:
    """The installed torch's folder (found, not imported)."""
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def built_for() -> str:
    """What the extension is built against and holds as a text, so that another torch's or Python's is told apart."""
    version = runpy.run_path(os.path.join(_torch(), "version.py"))["__version__"]
    return "torch %s, %s" % (version, sysconfig.get_config_var("SOABI"))


def _newer(target, sources) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in sources)


def _lib_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "csa2.h"), __file__])


def _bind_up_to_date() -> bool:
    if not _newer(BIND, [os.path.join(CSRC, "bind.cpp"), os.path.join(INCLUDE, "csa2.h"), __file__]):
        return False
    with open(BIND, "rb") as f:
        return built_for().encode() in f.read()


def up_to_date() -> bool:
    return _lib_up_to_date() and _bind_up_to_date()


def _build_bind():
    """The extension, against the installed torch."""
    torch = _torch()
    lib = os.path.join(torch, "lib")
    tmp = BIND + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", '-DCSA2_BUILT_FOR="%s"' % built_for(),
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch, "include"), os.path.join(CSRC, "bind.cpp"), "-o", tmp, "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("bind.cpp: %s%s" % (r.stdout, r.stderr))
    os.replace(tmp, BIND)


def _bring_bind(force):
    """The package works without the extension: what keeps it from being built is said, and a stale one goes."""
    try:
        if force or not _bind_up_to_date():
            _build_bind()
    except Exception as e:
        if os.path.exists(BIND):
            os.remove(BIND)
        sys.stderr.write("%s is not built, calls will take some microseconds longer: %s\n" % (os.path.basename(BIND), e))


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and _lib_up_to_date():
        _bring_bind(False)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        bind = ex.submit(_bring_bind, force)
        objs = list(ex.map(compile_one, sources()))
        bind.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=(["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])))
