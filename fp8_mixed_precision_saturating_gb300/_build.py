"""Build libfp8gb.so in-tree with nvcc for sm_103a (one translation unit per job, in parallel)."""
from __future__ import annotations

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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp8gb.so")
# (named for this interpreter: another one does not import it)
FASTCALL = os.path.join(PKG, "_fastcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
FASTCALL_SOURCE = os.path.join(CSRC, "fastcall.c")
SOURCES = ["api.cu", "quant.cu", "gemm.cu", "api4.cu", "quant4.cu", "gemm4.cu", "norm_fwd.cu", "norm_fwd_ring.cu", "norm_bwd.cu", "norm_bwd_ring.cu", "api_heads.cu", "qk_rope.cu", "kv_append.cu", "paged_attention.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfp8gb.so")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "fastcall.c"]
    files.append(os.path.join(INCLUDE, "fp8gb.h"))
    files.append(os.path.abspath(__file__))
    return files


def python_header() -> str | None:
    """The folder of Python.h, where the host has it and a C compiler."""
    d = sysconfig.get_paths()["include"]
    return d if os.path.exists(os.path.join(d, "Python.h")) and shutil.which("gcc") else None


def build_fastcall(force: bool = False) -> bool:
    """_fastcall: the binding's calls in C. Without Python.h, or where it does not compile (it needs Python 3.10), the ctypes
    wrappers are used alone."""
    untagged = os.path.join(PKG, "_fastcall.so")  # an older build's, which any interpreter would import
    if untagged != FASTCALL and os.path.exists(untagged):
        os.remove(untagged)
    include = python_header()
    if include is None:
        return False
    if not force and _newer(FASTCALL, [FASTCALL_SOURCE, os.path.join(INCLUDE, "fp8gb.h"), os.path.abspath(__file__)]):
        return True
    tmp = FASTCALL + ".tmp"
    r = subprocess.run(["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I", include, "-I", INCLUDE, FASTCALL_SOURCE, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(FASTCALL):  # made from another source
            os.remove(FASTCALL)
        warnings.warn(f"fastcall.c did not compile; calls go through ctypes:\n{r.stdout}\n{r.stderr}", RuntimeWarning, stacklevel=2)
        return False
    os.replace(tmp, FASTCALL)
    return True


def _newer(path, sources) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in sources)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link libfp8gb.so. Returns its path."""
    if not force and up_to_date():
        build_fastcall()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *CFLAGS, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        log = os.path.join(BUILD, src.replace(".cu", ".ptxas.txt"))
        with open(log, "w") as f:
            f.write(r.stdout + r.stderr)
        if verbose:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    build_fastcall(force=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
