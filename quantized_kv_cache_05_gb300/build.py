"""Build the CUDA library libkvq.so (nvcc, sm_103a only) and the marshalling
module of the per-step calls (the C compiler, CPython headers) in-tree."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkvq.so")
CALL = os.path.join(HERE, "_kvq_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
SOURCES = ["kvq_api.cu", "kvq_append.cu", "kvq_decode.cu", "kvq_decode_nvfp4.cu", "kvq_mla.cu",
           "kvq_prefill.cu", "kvq_rope.cu",
           "kvq_shared.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# host code: no FP contraction (the host-side checks emulate device fp32
# operations one by one)
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-ffp-contract=off",
         "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkvq.so")
    return p


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "kvq.h"))
    return max(os.path.getmtime(f) for f in files)


def build_call() -> str:
    """The marshalling module of runtime.py's per-step calls (_kvq_call)."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        raise RuntimeError("no C compiler: it is required to build the _kvq_call module")
    tmp = CALL + ".tmp"
    cmd = [cc, "-O2", "-Wall", "-Wextra", "-shared", "-fPIC", "-std=c11", "-I", INCLUDE, "-I",
           sysconfig.get_paths()["include"], "-o", tmp, os.path.join(CSRC, "kvq_call.c")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cc} failed for kvq_call.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)
    return CALL


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= _deps_mtime()
                         for f in (LIB, CALL)):
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    extra = extra or []

    def compile_one(src: str) -> str:
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        call = ex.submit(build_call)
        objs = list(ex.map(compile_one, SOURCES))
        call.result()
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    build(force=True, verbose=True, extra=sys.argv[1:])
    print(LIB)
