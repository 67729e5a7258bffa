"""Build the sm_103a shared library in-tree with nvcc (no cmake, no torch), and, where
PyTorch is installed, the compiled part of the cache operators' Python binding (g++,
PyTorch's headers).

    python -m exact_attention_63_gb300.build

Compiles the translation units in parallel and links
``exact_attention_63_gb300/libattn_gb300.so`` and ``_cache_bind.so`` beside it.  The library is linked
against the shared CUDA runtime so it uses the same runtime instance as the
host process (PyTorch loads ``libcudart.so.13`` too).
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libattn_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SOURCES = ["attn_api.cu", "attn_static.cu", "attn_fwd_d64.cu", "attn_fwd_d64_causal.cu", "attn_fwd_d128.cu",
           "attn_fwd_d128_causal.cu", "attn_bwd.cu", "attn_fwd_fp8.cu", "cache_api.cu", "cache_attn.cu", "cache_weights.cu",
           "cache_evict.cu", "cache_fp8.cu", "cache_attn_fp8.cu",
           "cache_attn_fp8_wide.cu", "cache_pages.cu", "rotary.cu"]
BIND_SOURCE = "cache_bind.cpp"
BIND_PATH = os.path.join(PKG, "_cache_bind.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin directory on PATH)")


def cuda_home(nvcc: str) -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))


def compile_flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC,
                   *extra]


def run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stdout.write(r.stdout + r.stderr)


def torch_dir():
    """Where PyTorch (with CUDA) is installed, or None."""
    spec = importlib.util.find_spec("torch")
    for path in (spec.submodule_search_locations or []) if spec else []:
        if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")):
            return path
    return None


def compile_bind(torch, cuda, verbose=False):
    """Object of the binding against the PyTorch in `torch` and the toolkit in `cuda`."""
    obj = os.path.join(BUILD_DIR, "cache_bind.o")
    inc = [sysconfig.get_paths()["include"], os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"), INCLUDE]
    run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", *("-I" + i for i in inc), "-c",
         os.path.join(CSRC, BIND_SOURCE), "-o", obj], f"compiler for {BIND_SOURCE}", verbose)
    return obj


def build(verbose: bool = False, extra_flags=()) -> str:
    """The library, which needs nvcc alone; then the binding, where PyTorch is installed.  What fails of
    the binding is raised when the library is in place."""
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = compile_flags(extra_flags)

    def one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        run([nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc for {src}", verbose)
        return obj

    home = cuda_home(nvcc)
    torch = torch_dir()
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bound = None if torch is None else ex.submit(compile_bind, torch, home, verbose)
        objs = list(ex.map(one, SOURCES))
    libdir = os.path.join(home, "lib64")
    tmp = LIB_PATH + ".tmp"
    run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-rpath," + libdir, "-o", tmp, *objs], "link")
    os.replace(tmp, LIB_PATH)
    if bound is None:
        print("no PyTorch with CUDA here: the cache operators' Python binding is not built", file=sys.stderr)
        return LIB_PATH
    # (torch's libraries are in the process before this one is loaded; it finds the
    # library above beside itself)
    tmp = BIND_PATH + ".tmp"
    run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, bound.result(), "-L" + os.path.join(torch, "lib"),
         "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-L" + PKG, "-lattn_gb300",
         "-Wl,-rpath,$ORIGIN"], "link of the binding")
    os.replace(tmp, BIND_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
