"""Build the CUDA library libpts_gemm.so in-tree with nvcc for sm_103a.

The translation units (the wide-tile 1-SM kernels, the 2-SM kernels, the
narrow-tile 1-SM and 2-SM kernels, the C ABI, the allocation-free entry point,
the tensor-pipe peak probe, and the expert layer's products, row kernels,
4-bit products and C ABI) are compiled in parallel, then linked with the static
CUDA runtime.  Nothing is rebuilt when the library is newer than every source
file.

The expert layer's Python calls are a CPython extension that links to the
library (build_experts()): a file of its own for every interpreter, built at
the first of these calls, so that everything else needs no Python headers.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libpts_gemm.so")
EXPERTS = os.path.join(LIBDIR, "pts_experts" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING = os.path.join(CSRC, "expert_binding.cpp")
UNITS = ["gemm_cg1.cu", "gemm_cg2.cu", "gemm_narrow.cu", "gemm_narrow_cg2.cu", "gemm_api.cu", "gemm_noalloc.cu",
         "peak_probe.cu", "expert_fwd.cu", "expert_dgrad.cu", "expert_wgrad.cu", "expert_route.cu", "nibble_f16.cu",
         "nibble_bf16.cu", "nibble_rows_f16.cu", "nibble_rows_bf16.cu", "expert_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpts_gemm.so")


def _sources():
    return ([f for f in glob.glob(os.path.join(CSRC, "*")) if f != BINDING]
            + [os.path.join(ROOT, "include", "pts_gemm.h"), os.path.abspath(__file__)])


def _newer(built, sources) -> bool:
    return os.path.exists(built) and all(os.path.getmtime(s) <= os.path.getmtime(built) for s in sources)


def up_to_date() -> bool:
    return _newer(LIB, _sources())


def experts_up_to_date() -> bool:
    # (the module reads the handle's struct: it goes with the library's sources)
    return _newer(EXPERTS, _sources() + [BINDING])


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    cc = nvcc()

    def compile_one(unit):
        obj = os.path.join(BUILD, unit.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, unit), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {unit}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(len(UNITS)) as ex:
        objs = list(ex.map(compile_one, UNITS))
    tmp = LIB + ".tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build_experts(force: bool = False) -> str:
    """The extension module (and the library first, if there is none; one that may be loaded is not replaced here)."""
    if not os.path.exists(LIB):
        build()
    if not force and experts_up_to_date():
        return EXPERTS
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        raise RuntimeError(f"{os.path.join(include, 'Python.h')} not found: the expert layer's calls from Python need the "
                           "interpreter's headers (the C ABI and the other calls do not)")
    tmp = EXPERTS + ".tmp"
    r = subprocess.run([nvcc(), *FLAGS, "-shared", "-I" + include, "-I" + os.path.join(ROOT, "include"), BINDING,
                        "-cudart", "none", "-L" + LIBDIR, "-lpts_gemm", "-Xlinker", "-rpath,$ORIGIN", "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"expert_binding.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXPERTS)
    return EXPERTS


if __name__ == "__main__":
    print(build(force=True, verbose=True))
