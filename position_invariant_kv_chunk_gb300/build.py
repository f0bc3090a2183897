"""Build the Kamera C-ABI shared library for sm_103a with nvcc (in-tree).

``build()`` compiles every ``csrc/*.cu`` translation unit in parallel with
``-gencode arch=compute_103a,code=sm_103a`` and links them into
``_build/libkamera.so``, and, against the installed torch's headers, the Python
binding of the decode-step entry points (``csrc/kamera_binding.cpp`` ->
``_build/_kamera_binding.so``).  Rebuilds only when a source or header is newer
than its library.  The library needs none of what the binding does (g++, Python's
and torch's headers): without it ``build()`` warns, the entry points that go through
ctypes work, and those of the binding raise its build error.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libkamera.so")
BINDING_SRC = os.path.join(CSRC, "kamera_binding.cpp")
BINDING_PATH = os.path.join(BUILD_DIR, "_kamera_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the Kamera CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(out: str) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_version() -> str:
    import torch
    return torch.__version__


def _binding_stale() -> bool:
    """Older than its source or the header, or built against another torch."""
    stamp = BINDING_PATH + ".torch"
    if not os.path.exists(BINDING_PATH) or not os.path.exists(stamp):
        return True
    t = os.path.getmtime(BINDING_PATH)
    if any(os.path.getmtime(d) > t for d in (BINDING_SRC, os.path.join(INCLUDE, "kamera.h"), os.path.abspath(__file__))):
        return True
    with open(stamp) as f:
        return f.read() != _torch_version()


def _compile_binding() -> str:
    """The binding's object file (needs nothing of libkamera.so but the header)."""
    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD_DIR, "kamera_binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"), "-isystem",
           os.path.join(root, "include", "torch", "csrc", "api", "include"), "-isystem", cuda, "-isystem",
           sysconfig.get_paths()["include"], "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(BINDING_SRC)}:\n{r.stderr[-4000:]}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", BUILD_DIR, "-lkamera", "-L", libs,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_PATH + ".torch", "w") as f:
        f.write(_torch_version())


def build_binding(force: bool = False) -> str:
    """Builds the Python binding where it is missing or stale (the library is there); raises where it cannot be."""
    if force or _binding_stale():
        os.makedirs(BUILD_DIR, exist_ok=True)
        _link_binding(_compile_binding())
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    lib = force or _stale(LIB_PATH)
    try:
        binding, why = force or _binding_stale(), None
    except ImportError as e:   # no torch: nothing to build it against
        binding, why = False, e
    if lib or binding:
        os.makedirs(BUILD_DIR, exist_ok=True)
        with ThreadPoolExecutor(max_workers=1) as ex:   # the binding compiles beside the library
            obj = ex.submit(_compile_binding) if binding else None
            if lib:
                _build_library(verbose, extra_flags)
            if obj is not None:
                try:
                    _link_binding(obj.result())
                except (ImportError, OSError, RuntimeError) as e:
                    why = e
                    if os.path.exists(BINDING_PATH):   # built from older sources
                        os.remove(BINDING_PATH)
    if why is not None:
        warnings.warn(f"the Kamera library is built, the Python binding of its decode-step entry points is not: {why}")
    return LIB_PATH


def _build_library(verbose: bool, extra_flags) -> str:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB_PATH + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
