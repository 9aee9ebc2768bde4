"""Build libmsa.so (the MSA C-ABI library) for sm_103a, and the compiled
Python binding ``_binding.so`` of the serving step's operators, in-tree.

Each CUDA translation unit under csrc/ is compiled by nvcc in parallel, then
linked into ``libmsa.so`` next to this file; ``csrc/binding.cpp`` is compiled
by g++ against torch's headers meanwhile and linked with ``libmsa.so``.
Each is rebuilt only when a source or header is newer than it, the binding
also when Python or torch is another than it was compiled for.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmsa.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
STAMP = os.path.join(OBJ, "binding.stamp")  # what the binding was compiled for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
           "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _fresh(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def _library_fresh() -> bool:
    return _fresh(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) + _headers())


def _installed() -> str:
    """What a compiled binding goes with: this Python and the installed torch."""
    import torch
    return f"{sys.version}\n{torch.__version__} {os.path.dirname(torch.__file__)}\n"


def _binding_fresh() -> bool:
    try:
        with open(STAMP) as f:
            if f.read() != _installed():
                return False
    except (OSError, ImportError):
        return False
    return _fresh(BINDING, [BINDING_SOURCE] + _headers())


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
    return _library_fresh() and _binding_fresh()


def _run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)


def _build_library(pool, verbose, extra):
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        _run([nvcc, *ARCH, *NVFLAGS, *extra, "-c", src, "-o", obj], f"nvcc for {src}", verbose)
        return obj

    objs = list(pool.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", *objs, "-o", tmp, "-lcudart_static", "-ldl", "-lpthread", "-lrt"], "link")
    os.replace(tmp, LIB)


def _compile_binding(verbose):
    obj = os.path.join(OBJ, "binding.cpp.o")
    _run(["g++", *_binding_flags()[0], "-c", BINDING_SOURCE, "-o", obj], f"g++ for {BINDING_SOURCE}", verbose)
    return obj


def _link_binding(obj):
    tmp = BINDING + f".tmp{os.getpid()}"
    _run(["g++", "-shared", obj, "-o", tmp, "-L", HERE, "-l:libmsa.so", *_binding_flags()[1],
          "-Wl,-rpath,$ORIGIN"], "link")
    os.replace(tmp, BINDING)
    with open(STAMP, "w") as f:
        f.write(_installed())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Builds what is out of date; returns the library's path.

    The library needs nvcc alone. The binding needs g++ and the headers of
    torch and Python too: where it cannot be built, that is a warning, and the
    calls that go through it raise.
    """
    library, binding = force or not _library_fresh(), force or not _binding_fresh()
    if not library and not binding:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    workers = max(2, min(8, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(1) as one, cf.ThreadPoolExecutor(workers - 1) as pool:
        bound = one.submit(_compile_binding, verbose) if binding else None
        if library:
            _build_library(pool, verbose, extra)
        if binding:
            try:
                _link_binding(bound.result())
            except Exception as e:  # a missing compiler, missing headers, another compiler's errors
                warnings.warn(f"_binding.so, the compiled calls of the serving step's operators, was not built: {e}",
                              RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force="--force" in sys.argv or bool(extra), verbose=v or bool(extra), extra=extra))
