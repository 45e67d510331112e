"""Build libmmq_gb300.so in-tree with nvcc for sm_103a (translation units compiled in parallel), and the C++ half of the
Python binding with the host compiler against the installed torch."""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libmmq_gb300.so")
PEAKS_LIB = os.path.join(LIBDIR, "libmmq_peaks.so")
PEAKS_SRC = os.path.join(PKG, "probe", "peaks.cu")
BIND_LIB = os.path.join(LIBDIR, "_attention.so")
BIND_SRC = os.path.join(PKG, "bind", "attention.cpp")
OBJDIR = os.path.join(ROOT, "_build", "obj")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "mmq.h")]


def _newer(lib, deps) -> bool:
    return os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in deps)


def _library_up_to_date() -> bool:
    return _newer(LIB, _deps()) and _newer(PEAKS_LIB, [PEAKS_SRC, os.path.join(ROOT, "include", "mmq_peaks.h")])


def _torch_version() -> str | None:
    """What a binding is compiled against (its C++ interface changes with the version), None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        return f"{spec.origin}\n{sys.version}\n{f.read()}"


def _stamp() -> str:
    return os.path.join(OBJDIR, "bind_attention.torch")


def _binding_up_to_date() -> bool:
    version = _torch_version()
    if version is None:
        return True                                           # nothing could load one
    if not _newer(BIND_LIB, [BIND_SRC, os.path.join(ROOT, "include", "mmq.h")]) or not os.path.exists(_stamp()):
        return False
    with open(_stamp()) as f:
        return f.read() == version


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr}")


def _bind_object():
    """Compile the binding: torch's and CUDA's headers, no CUDA code."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    obj = os.path.join(OBJDIR, "bind_attention.o")
    include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", *(f"-I{d}" for d in include), "-c", BIND_SRC, "-o",
          obj], f"c++ failed for {BIND_SRC}")
    return obj, os.path.join(torch_dir, "lib")


def _link_binding(obj, torch_lib):
    tmp = BIND_LIB + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{torch_lib}", "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-lc10_cuda", f"-L{LIBDIR}", "-lmmq_gb300", "-Wl,-rpath,$ORIGIN"], "link of the binding failed")
    os.replace(tmp, BIND_LIB)
    with open(_stamp(), "w") as f:
        f.write(_torch_version())


def build(force: bool = False, verbose: bool = False) -> str:
    """Both libraries, then the binding: the C library needs neither torch nor Python's headers, and is there where
    compiling the binding fails (which raises) or there is no torch to bind to."""
    library = force or not _library_up_to_date()
    binding = _torch_version() is not None and (force or not _binding_up_to_date())
    if not library and not binding:
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC, *ARCH, *CFLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        _run(cmd, f"nvcc failed for {src}")
        return obj

    def link(objs, lib):
        tmp = lib + f".tmp{os.getpid()}"
        _run([NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"], "link failed")
        os.replace(tmp, lib)

    with ThreadPoolExecutor(max_workers=max(4, os.cpu_count() or 4)) as ex:
        bind = ex.submit(_bind_object) if binding else None
        if library:
            *objs, peaks_obj = ex.map(compile_one, sources() + [PEAKS_SRC])
            link([peaks_obj], PEAKS_LIB)
            link(objs, LIB)
    if bind:
        _link_binding(*bind.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
