"""Build libokv.so in-tree: every CUDA source for sm_103a, compiled in parallel, linked shared; and _calls.so,
the Python calls that read torch tensors, for the torch that is installed. Where those cannot be built the
library is built without them, and their first use raises ImportError.

Run as ``python -m sparse_kv_cache_draft_gb300.build`` or through ``__graft_entry__.build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libokv.so")
CALLS = os.path.join(HERE, "_calls.so")
CXX = os.environ.get("CXX", "g++")
BUILD_DIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["okv_api.cu", "k_summary.cu", "k_select.cu", "k_gather.cu", "k_attend.cu", "k_rows.cu", "k_tree.cu", "k_chunk.cu",
           "k_chunk_f32.cu", "k_weigh.cu", "k_evict.cu"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the okv CUDA library cannot be built")


def _flags(verbose: bool):
    f = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(HERE, "..", "include")] + ARCH
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    deps = [src, os.path.join(HERE, "..", "include", "okv.h")] + [
        os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return any(os.path.getmtime(d) > os.path.getmtime(obj) for d in deps)


def _build_calls(nv: str, force: bool) -> str:
    """Compile py_calls.cpp for the Python and torch there are, where its object is not of these sources and those."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    made_for = f"{sysconfig.get_config_var('SOABI')} torch {importlib.metadata.version('torch')}\n"
    src, obj, tag = os.path.join(CSRC, "py_calls.cpp"), os.path.join(BUILD_DIR, "py_calls.o"), os.path.join(BUILD_DIR, "py_calls.for")
    if not force and os.path.exists(tag) and open(tag).read() == made_for and not _stale(obj, src):
        return obj
    include = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nv))), "include")]
    tmp = f"{obj}.tmp{os.getpid()}"
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-I", os.path.join(HERE, "..", "include")] +
         [a for d in include for a in ("-isystem", d)] + ["-c", src, "-o", tmp], "the compiler for py_calls.cpp")
    os.replace(tmp, obj)
    with open(tag, "w") as f:
        f.write(made_for)
    return obj


def _link_calls(obj: str) -> None:
    if os.path.exists(CALLS) and os.path.getmtime(CALLS) >= os.path.getmtime(obj):
        return
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    tmp = CALLS + f".tmp{os.getpid()}"
    _run([CXX, "-shared", obj, "-o", tmp, "-L", HERE, "-l:libokv.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(torch_dir, "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], "link of _calls.so")
    os.replace(tmp, CALLS)


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")
    return r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    nv = nvcc()
    jobs = []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD_DIR, s.replace(".cu", ".o"))
        if force or verbose or _stale(obj, src):
            jobs.append(([nv] + _flags(verbose) + ["-c", src, "-o", obj], f"nvcc for {src}"))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        calls = ex.submit(_build_calls, nv, force) if importlib.util.find_spec("torch") else None
        for log in ex.map(lambda job: _run(*job), jobs):
            if verbose and log:
                sys.stderr.write(log)
    objs = [os.path.join(BUILD_DIR, s.replace(".cu", ".o")) for s in SOURCES]
    if jobs or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        _run([nv] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcuda"], "link of libokv.so")
        os.replace(tmp, LIB)
    if calls is not None:
        try:
            _link_calls(calls.result())
        except (RuntimeError, OSError, ImportError) as e:  # no compiler, headers or package data of torch
            if os.path.exists(CALLS):
                os.remove(CALLS)
            sys.stderr.write(f"libokv.so is built; norm_rope, append_qkv_static, attend_tree_static, attend_chunk_static, evict_static and Rotary are not:\n{e}\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
