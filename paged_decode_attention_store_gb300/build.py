"""Build libpagedkv.so in-tree (nvcc for sm_103a, g++ for the host bookkeeping).

Objects go to ``_build/`` next to this file; the library to
``libpagedkv.so`` next to this file, and the binding's argument marshalling
(``csrc/python/marshal.cpp``, against Python's and torch's headers) to
``_marshal.so``. Translation units compile in parallel
and only when a source or header is newer than the library.
``build_traced()`` builds the tracing variant of the prefill kernel
(``-DKVP_PREFILL_TRACE``) as ``libpagedkv_trace.so`` from objects in
``_build/trace/``; it is a measuring tool, never the product.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpagedkv.so")
TRACE_LIB = os.path.join(HERE, "libpagedkv_trace.so")
MARSHAL_SRC = os.path.join(CSRC, "python", "marshal.cpp")
MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_FOR = os.path.join(BUILD, "marshal_for")  # the torch and Python that it was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu"))) + sorted(glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in _deps())


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("build step failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def marshal_for() -> str:
    """The torch and Python whose headers' layouts the marshalling takes for granted."""
    import torch

    return f"torch {torch.__version__} Python {sys.version_info[0]}.{sys.version_info[1]}"


def marshal_is_new() -> bool:
    if not (os.path.exists(MARSHAL) and os.path.exists(MARSHAL_FOR)):
        return False
    with open(MARSHAL_FOR) as f:
        return f.read() == marshal_for() and os.path.getmtime(MARSHAL) > os.path.getmtime(MARSHAL_SRC)


def build_marshal(force: bool = False) -> str:
    """Compile the binding's argument marshalling; returns its path."""
    if not force and marshal_is_new():
        return MARSHAL
    import sysconfig

    import torch

    os.makedirs(BUILD, exist_ok=True)
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = MARSHAL + ".tmp"
    _run(["g++", "-O2", "-std=c++20", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], "-I", os.path.join(home, "include"),
          "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DKVP_BUILT_FOR="{marshal_for()}"',
          MARSHAL_SRC, "-o", tmp,
          "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
          "-Wl,-rpath," + os.path.join(home, "lib")])
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_FOR, "w") as f:
        f.write(marshal_for())
    return MARSHAL


def build(force: bool = False, verbose: bool = False, lib: str = LIB, objdir: str = BUILD,
          defines: tuple = ()) -> str:
    """Compile every translation unit and link ``lib`` (libpagedkv.so by
    default, the argument marshalling beside it); returns its path."""
    if not force and not needs_build(lib):
        if lib == LIB:
            build_marshal()
        return lib
    os.makedirs(objdir, exist_ok=True)
    nvcc = _nvcc()
    jobs = []
    for src in _sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        if src.endswith(".cu"):
            cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                   *[f"-D{d}" for d in defines], "-Xptxas", "-v", "-c", src, "-o", obj]
        else:
            cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-c", src, "-o", obj]
        jobs.append((cmd, obj))
    with ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
        marshal = ex.submit(build_marshal, force) if lib == LIB else None
        logs = list(ex.map(lambda j: _run(j[0]), jobs))
        if marshal:
            marshal.result()
    if verbose:
        for log in logs:
            sys.stdout.write(log)
    tmp = lib + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *[o for _, o in jobs], "-o", tmp])
    os.replace(tmp, lib)
    return lib


def build_traced(force: bool = False) -> str:
    """The tracing variant of the library (the prefill kernel's stamps on)."""
    return build(force=force, lib=TRACE_LIB, objdir=os.path.join(BUILD, "trace"), defines=("KVP_PREFILL_TRACE",))


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
