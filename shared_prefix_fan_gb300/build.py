"""Builds libfanout.so in-tree with nvcc for sm_103a (no cmake, no torch).

Translation units are compiled in parallel, then linked into one shared
library: lib/libfanout.so next to this file. Beside it lib/_host_calls, the extension module
of the small serving calls' host side (the C compiler, this interpreter's headers; it is
named after the interpreter it was built for). Without those the library is built all the
same, and only the calls that need the module raise.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "libfanout.so")
HOST = os.path.join(LIBDIR, "_host_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
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


def _host_calls(srcs) -> None:
    gcc, headers = shutil.which("gcc"), sysconfig.get_paths()["include"]
    if not gcc or not os.path.exists(os.path.join(headers, "Python.h")):
        warnings.warn(f"_host_calls is not built ({'no Python.h in ' + headers if gcc else 'no gcc'}): "
                      "the calls of the 8-bit cache and of drafted trees will raise")
        if os.path.exists(HOST) and not _current(HOST, srcs):
            os.remove(HOST)  # of other sources
        return
    tmp = HOST + ".tmp"
    cmd = [gcc, "-O2", "-fPIC", "-shared", "-Wall", "-I", headers,
           os.path.join(CSRC, "host_calls.c"), "-o", tmp, "-L", LIBDIR, "-l:libfanout.so",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host_calls.c failed:\n{r.stderr}")
    os.replace(tmp, HOST)


def _current(built: str, srcs) -> bool:
    return os.path.exists(built) and os.path.getmtime(built) >= max(os.path.getmtime(s) for s in srcs)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link; skips what is newer than every source of its own."""
    header = os.path.join(os.path.dirname(HERE), "include", "fanout.h")
    srcs = [os.path.join(CSRC, s) for s in SOURCES] + [
        os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    if force or not _current(LIB, srcs + [header]):
        _library(verbose_ptxas)
    host_srcs = [os.path.join(CSRC, "host_calls.c"), header]
    if force or not _current(HOST, host_srcs):
        _host_calls(host_srcs)
    return LIB


def _library(verbose_ptxas: bool) -> None:
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
    if verbose_ptxas:
        print("".join(logs))


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas=True))
