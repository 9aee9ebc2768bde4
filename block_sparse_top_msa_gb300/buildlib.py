"""Build libmsa.so (the MSA C-ABI library) for sm_103a, and the compiled
Python binding ``_binding.so`` of the serving step's operators, in-tree.

Each CUDA translation unit under csrc/ is compiled by nvcc in parallel, then
linked into ``libmsa.so`` next to this file; ``csrc/binding.cpp`` is compiled
by g++ against torch's headers meanwhile and linked with ``libmsa.so``.
Rebuilds only when a source or header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmsa.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
           "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cpp")) +
            glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def _binding_flags():
    """g++ flags for a module against the installed torch: (compile, link)."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    return (["-O2", "-std=c++17", "-fPIC", "-I", inc,
             "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
             "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"],
            ["-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
             "-lc10"])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    nvcc = _nvcc()

    compile_flags, link_flags = _binding_flags()
    binding = os.path.join(CSRC, "binding.cpp")

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        if src == binding:
            cmd = ["g++", *compile_flags, "-c", src, "-o", obj]
        else:
            cmd = [nvcc, *ARCH, *NVFLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        bound, *objs = ex.map(compile_one, [binding] + sources())
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", *objs, "-o", tmp, "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", bound, "-o", tmp, "-L", HERE, "-l:libmsa.so", *link_flags,
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force="--force" in sys.argv or bool(extra), verbose=v or bool(extra), extra=extra))
