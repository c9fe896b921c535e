"""Build libmpm.so and its torch binding in-tree (nvcc for sm_103a and g++; no
cmake).

Each .cu file compiles to an object in parallel; the objects link into
``microscaled_precision_moe_gb300/libmpm.so``, for which nvcc is enough.
``csrc/binding.cpp``, which marshals torch tensors into some of the library's
calls, compiles beside them against the headers of the running torch and links
into ``_binding.so``; without torch there is none, and where its build fails the
library is still there.  Rebuilds what a source or header is newer than, and the
binding for another torch or Python.

    python -m microscaled_precision_moe_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

from ._lib import binding_abi

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmpm.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "binding_for.txt")     # the torch and Python it was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
              "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _older(target: str, files) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in files)


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def library_needs_build() -> bool:
    return _older(LIB, _sources() + _headers() + [__file__])


def _built_for() -> str:
    try:
        with open(BINDING_FOR) as f:
            return f.read()
    except OSError:
        return ""


def binding_needs_build() -> bool:
    return has_torch() and (_older(BINDING, _headers() + [BINDING_SRC, __file__]) or _built_for() != binding_abi())


def needs_build() -> bool:
    return library_needs_build() or binding_needs_build()


def _run(cmd, what: str, verbose: bool = False):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)


def _compile(src: str, verbose: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    _run([nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj], f"nvcc {src}", verbose)
    return obj


def _compile_binding(verbose: bool) -> str:
    from torch.utils.cpp_extension import include_paths
    import torch
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    obj = os.path.join(BUILD, "binding.cpp.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f'-DMPM_BINDING_FOR="{binding_abi()}"',
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          "-I", os.path.join(ROOT, "include"), *[f for p in inc for f in ("-isystem", p)],
          "-c", BINDING_SRC, "-o", obj], f"g++ {BINDING_SRC}", verbose)
    return obj


def _link_binding(obj: str) -> None:
    from torch.utils.cpp_extension import library_paths
    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libmpm.so",
          *[f for p in library_paths() for f in ("-L", p)], "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "link of _binding.so")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(binding_abi())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Build what is out of date, or everything: the library's path.  An error
    of the binding is raised after the library is in place."""
    library = force or library_needs_build()
    binding = has_torch() and (force or binding_needs_build())
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources() if library else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding_obj = ex.submit(_compile_binding, verbose) if binding else None
        objs = list(ex.map(lambda s: _compile(s, verbose, list(extra)), srcs))
        if library:
            tmp = LIB + ".tmp"
            _run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], "link of libmpm.so")
            os.replace(tmp, LIB)
        if binding:
            _link_binding(binding_obj.result())
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register/smem usage")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_v else []
    print(build(force=a.force or a.ptxas_v, verbose=a.verbose or a.ptxas_v, extra=extra))


if __name__ == "__main__":
    sys.exit(main())
