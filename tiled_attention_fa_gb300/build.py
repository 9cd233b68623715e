"""Build the C-ABI shared library in-tree with nvcc (sm_103a only).

    python -m tiled_attention_fa_gb300.build          # builds libfa_gb300.so next to this file

Each .cu unit compiles in parallel to an object file under ``_build/``; the
objects then link into ``libfa_gb300.so`` with the CUDA runtime linked
statically, so loading the library needs no GPU and no libcuda at load time.
``_binding.so``, the part of the Python binding that works on torch tensors in
C++, compiles alongside against the installed torch and links to the library.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB_NAME = "libfa_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
UNITS = ["api.cu", "fwd.cu", "bwd.cu", "decode.cu", "paged.cu", "weights.cu", "evict.cu"]
BINDING_PATH = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def _flags(verbose_ptxas: bool) -> list:
    f = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _compile(unit: str, verbose_ptxas: bool) -> tuple:
    src = os.path.join(CSRC, unit)
    obj = os.path.join(BUILD, unit.replace(".cu", ".o"))
    cmd = [nvcc(), "-c", src, "-o", obj] + _flags(verbose_ptxas)
    r = subprocess.run(cmd, capture_output=True, text=True)
    return unit, obj, r.returncode, r.stdout + r.stderr


def _compile_binding() -> tuple:
    """binding.cpp against the installed torch (headers only are needed here)."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [os.environ.get("CXX", "g++"), "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj, "-O2",
           "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", inc, "-I",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda, "-I",
           sysconfig.get_paths()["include"]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return "binding.cpp", obj, r.returncode, r.stdout + r.stderr


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L" + HERE, "-l:" + LIB_NAME,
           "-Wl,-rpath,$ORIGIN", "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of the binding failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, BINDING_PATH)


def build(verbose_ptxas: bool = False, quiet: bool = False) -> str:
    """Compile every unit and link the shared library; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(UNITS) + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda u: _compile(u, verbose_ptxas), UNITS))
        binding = binding.exception() or binding.result()
    failed = [r for r in results if r[2] != 0]
    for unit, _, rc, out in results:
        if (rc != 0 or verbose_ptxas) and out.strip():
            print(f"---- {unit} (rc={rc})\n{out}", file=sys.stderr)
    if failed:
        raise RuntimeError("nvcc failed for " + ", ".join(r[0] for r in failed))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), "-shared", "-Xlinker", "-soname=" + LIB_NAME, "-o", tmp] + [r[1] for r in results] + ARCH + \
        ["-Xcompiler", "-fPIC", "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB_PATH)
    # The C library stands by now: it needs nvcc alone, the binding torch's and
    # Python's headers too.  Where that fails, no binding of an earlier build stays
    # beside a library it may not fit.
    try:
        if isinstance(binding, BaseException):
            raise RuntimeError("the binding was not compiled (the library was)") from binding
        if binding[2] != 0:
            raise RuntimeError("the binding failed to compile (the library did compile):\n" + binding[3])
        _link_binding(binding[1])
    except RuntimeError:
        if os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)
        raise
    if not quiet:
        print("built", LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose_ptxas="-v" in sys.argv)
