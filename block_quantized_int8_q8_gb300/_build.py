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


def up_to_date() -> bool:
    for lib, deps in ((LIB, _deps()), (PEAKS_LIB, [PEAKS_SRC, os.path.join(ROOT, "include", "mmq_peaks.h")]),
                      (BIND_LIB, [BIND_SRC, os.path.join(ROOT, "include", "mmq.h")])):
        if not os.path.exists(lib):
            return False
        t = os.path.getmtime(lib)
        if any(os.path.getmtime(d) > t for d in deps):
            return False
    return True


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


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC, *ARCH, *CFLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=max(4, os.cpu_count() or 4)) as ex:
        bind = ex.submit(_bind_object)
        objs = list(ex.map(compile_one, sources() + [PEAKS_SRC]))
        bind_obj, torch_lib = bind.result()
    peaks_obj = objs.pop()
    tmp = PEAKS_LIB + f".tmp{os.getpid()}"
    r = subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, peaks_obj, "-lcudart"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, PEAKS_LIB)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = BIND_LIB + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, bind_obj, f"-L{torch_lib}", "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-lc10_cuda", f"-L{LIBDIR}", "-lmmq_gb300", "-Wl,-rpath,$ORIGIN"], "link of the binding failed")
    os.replace(tmp, BIND_LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
