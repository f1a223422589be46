"""Builds libfanout.so in-tree with nvcc for sm_103a (no cmake, no torch).

Translation units are compiled in parallel, then linked into one shared
library: lib/libfanout.so next to this file. Beside it lib/_host_calls.so, the extension
module of the small serving calls' host side (gcc, this interpreter's headers).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "libfanout.so")
HOST = os.path.join(LIBDIR, "_host_calls.so")
SOURCES = ["attn_fwd.cu", "lse_merge.cu", "kv_append.cu", "fanout_api.cu", "plan.cpp",
           "runtime.cpp", "fanout_noalloc.cu", "read_floor.cu", "tables.cu", "kv_q4.cu",
           "rows_api.cpp", "attn_rows.cu", "attn_rows_q8.cu", "attn_tree.cu", "kv_q8.cu", "tree.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler",
              "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, obj: str, verbose_ptxas: bool) -> str:
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose_ptxas and src.endswith(".cu"):
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    return r.stderr


def _host_calls() -> None:
    tmp = HOST + ".tmp"
    cmd = [shutil.which("gcc") or "gcc", "-O2", "-fPIC", "-shared", "-Wall",
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "host_calls.c"), "-o", tmp,
           "-L", LIBDIR, "-l:libfanout.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host_calls.c failed:\n{r.stderr}")
    os.replace(tmp, HOST)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link; skips work when the library is newer than every source."""
    srcs = [os.path.join(CSRC, s) for s in SOURCES] + [
        os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh", ".c"))]
    srcs.append(os.path.join(os.path.dirname(HERE), "include", "fanout.h"))
    if not force and os.path.exists(LIB) and os.path.exists(HOST):
        newest = max(os.path.getmtime(s) for s in srcs)
        if min(os.path.getmtime(LIB), os.path.getmtime(HOST)) >= newest:
            return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    objs = [os.path.join(objdir, s + ".o") for s in SOURCES]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        logs = list(ex.map(lambda a: _compile(*a, verbose_ptxas), zip(SOURCES, objs)))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _host_calls()
    if verbose_ptxas:
        print("".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas=True))
