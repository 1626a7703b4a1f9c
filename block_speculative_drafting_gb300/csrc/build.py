"""Build libdflash.so for sm_103a with nvcc (no cmake, no torch in it).

Usage: python -m block_speculative_drafting_gb300.csrc.build [--verbose]
Each .cu compiles on its own thread; the objects link into
block_speculative_drafting_gb300/libdflash.so (CUDA runtime linked
statically, so the library loads without a GPU).  binding.cpp, the compiled half
of target.py, becomes a Python extension beside it, against the installed torch.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
ROOT = os.path.dirname(PKG)
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdflash.so")
BINDING = os.path.join(PKG, "_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
BOUND_FOR = os.path.join(BUILD, "binding.txt")
SOURCES = ["api.cu", "k_quant.cu", "k_gemm.cu", "k_layer.cu", "k_stream.cu", "k_tc.cu", "k_tc_pair.cu",
           "k_attn_tc.cu", "ops.cu", "k_paged_append.cu", "k_paged_attn.cu", "k_paged_attn_tc.cu", "k_paged_attn4.cu",
           "k_paged_weights.cu", "k_paged_weights_few.cu",
           "k_paged_evict.cu", "k_verify.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _needs(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _text(path: str):
    try:
        with open(path) as f:
            return f.read()
    except FileNotFoundError:
        return None


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(HERE, f) for f in os.listdir(HERE) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "dflash.h"))
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src: str) -> str:
        path = os.path.join(HERE, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or _needs(obj, [path] + headers):
            cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", path, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
            if verbose:
                sys.stderr.write(r.stderr)
        return obj

    def compile_binding() -> None:
        src = os.path.join(HERE, "binding.cpp")
        torch = os.path.dirname(importlib.util.find_spec("torch").origin)
        cuda = os.path.dirname(os.path.dirname(shutil.which(nvcc()) or "/usr/local/cuda/bin/nvcc"))
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
               "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(cuda, "include"),
               "-isystem", sysconfig.get_path("include"), src, "-o", BINDING, "-L" + os.path.join(torch, "lib"),
               "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + os.path.join(torch, "lib")]
        # what it was built for: another torch has another ABI, and neither its name nor file times say so
        with open(os.path.join(torch, "version.py")) as f:
            made_for = "\n".join(cmd) + "\n" + f.read()
        if force or _needs(BINDING, [src] + headers) or _text(BOUND_FOR) != made_for:
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"{cmd[0]} failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
            with open(BOUND_FOR, "w") as f:
                f.write(made_for)

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        bound = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        bound.result()
    if force or _needs(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
