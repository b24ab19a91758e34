"""Build libmoe.so in-tree with nvcc for sm_103a (no cmake, no torch).

Each .cu file compiles to an object in parallel, then one shared-library link.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "lib", "libmoe.so")
# (named for the interpreter whose headers it is compiled with)
PYCALL = os.path.join(HERE, "lib", "_pycall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
SOURCES = ["moe_api.cu", "route.cu", "permute.cu", "ffn_decode.cu", "ffn_prefill.cu",
           "ffn_mxfp4act.cu", "ffn_fp8x2.cu", "linear_mxfp4.cu", "layer_few.cu",
           "moe_noalloc.cu", "route_grouped.cu", "lora.cu", "lora_prompt.cu",
           "combine_norm.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: libmoe needs the CUDA toolkit to build")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "moe.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def build_pycall(force: bool = False) -> str:
    """The CPython wrappers of the binding (pycall.c), with the system's C compiler."""
    src = os.path.join(CSRC, "pycall.c")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(ROOT, "include", "moe.h")))
    if not force and os.path.exists(PYCALL) and os.path.getmtime(PYCALL) >= newest:
        return PYCALL
    os.makedirs(os.path.dirname(PYCALL), exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = PYCALL + f".tmp{os.getpid()}"
    r = subprocess.run([os.environ.get("CC", "gcc"), "-O2", "-std=c11", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"],
                        "-I", cuda, src, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the C compiler failed on pycall.c:\n{r.stderr}")
    os.replace(tmp, PYCALL)
    return PYCALL


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    try:
        build_pycall(force)
    except (OSError, RuntimeError) as e:
        # the binding then makes these calls through ctypes; wrappers of older sources are not to be loaded
        with contextlib.suppress(FileNotFoundError):
            os.unlink(PYCALL)
        warnings.warn(f"pycall.c was not built, three calls take 3 us more each: {e}", RuntimeWarning, stacklevel=2)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
