"""Build the C-ABI library ``_lib/libgemm.so`` with nvcc for sm_103a.

Each translation unit compiles in parallel; the shared library links against
the CUDA runtime only (driver entry points are resolved at run time).  Beside
it, ``_lib/_binding.*.so``: the part of the Python binding that is in C, which
the serving operators' calls go through and nothing else does.  Where it cannot
be built (no headers of Python's), the library is built all the same.  Run as
``python layout_general_tensor_gb300/build.py`` or call :func:`build` (the
package itself loads the built library on import, so this file is loaded by
path).
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libgemm.so")
# (named for the interpreter that it is built for; another one does not find it)
BINDING = os.path.join(OUT_DIR, "_binding" + importlib.machinery.EXTENSION_SUFFIXES[0])
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["api.cu", "api_int4.cu", "gemm_tc.cu", "gemm_tc_pair.cu", "gemm_int4.cu", "gemm_int4_f8.cu",
           "aux_kernels.cu", "noalloc.cu", "reduce.cu", "attention.cu", "rope.cu", "prompt.cu", "cache.cu", "cache_attend.cu",
           "row_groups.cu", "gemm_grouped.cu", "adapters.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def nvcc_path():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _binding_deps():
    files = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return [*files, os.path.join(CSRC, "binding.c"), os.path.abspath(__file__)]


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.c"]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _up_to_date(target, deps):
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in deps)


def _build_binding(nvcc):
    """The binding's part in C; one that cannot be built is said on stderr and none is left."""
    include = [os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"), sysconfig.get_paths()["include"], INCLUDE]
    cmd = [shutil.which("gcc") or "cc", "-O2", "-Wall", "-fPIC", "-shared", *(f"-I{d}" for d in include),
           os.path.join(CSRC, "binding.c"), "-o", BINDING + ".tmp"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = f"{r.stdout}\n{r.stderr}" if r.returncode != 0 else None
    except OSError as e:
        failed = str(e)
    if failed is None:
        os.replace(BINDING + ".tmp", BINDING)
        return
    if os.path.exists(BINDING):
        os.remove(BINDING)
    print(f"binding.c does not compile, so the serving operators have no Python calls:\n{failed}", file=sys.stderr)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if anything changed) and return the library path."""
    binding = force or not _up_to_date(BINDING, _binding_deps())
    if not force and _up_to_date(LIB, _deps()):
        if binding:
            _build_binding(nvcc_path())
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = nvcc_path()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if (verbose or ptxas_info) and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bound = ex.submit(_build_binding, nvcc) if binding else None
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if bound:
        bound.result()
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    print(build(force=force, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv))
