"""Compile libtqd.so for sm_103a with nvcc (in-tree, under _build/).

Each translation unit is compiled in parallel, then linked into one shared
library with a plain C ABI (include/tqd.h).  No fast-math: the kernels call
expf / rsqrtf as specified by CUDA, never approximations enabled behind the
caller's back.
"""
from __future__ import annotations

import os
import runpy
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from importlib import util

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libtqd.so")
CALL = os.path.join(BUILD, "_tqd_call.so")
CALL_FOR = CALL + ".for"  # which torch and Python it was compiled against
SYNTH_SRC = os.path.join(ROOT, "synth", "tqd_synth.c")

SOURCES = ["tqd_kernels.cu", "tqd_persist.cu", "tqd_persist_bf16.cu", "tqd_engine.cu", "tqd_ops.cu", "tqd_noalloc.cu", "tqd_batch.cu",
           "tqd_sample.cu", "tqd_q4_cache.cu", "tqd_q4_attention.cu", "tqd_q4_matvec.cu", "tqd_logprobs.cu",
           "tqd_i8_rows.cu", "tqd_i8_matmul.cu", "tqd_rope_rows.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps_mtime() -> float:
    t = 0.0
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            t = max(t, os.path.getmtime(os.path.join(d, f)))
    return max(t, os.path.getmtime(__file__), os.path.getmtime(SYNTH_SRC))


def _torch() -> str | None:
    """Where torch is installed: the call module is built against it, and left out where there is none (or one without CUDA,
    which has not the libraries that it is linked with)."""
    spec = util.find_spec("torch")
    where = spec and list(spec.submodule_search_locations)[0]
    return where if where and os.path.exists(os.path.join(where, "lib", "libc10_cuda.so")) else None


def call_made_for(torch_version: str) -> str:
    """What a call module compiled now is for: it reads tensors by torch's own layout, so no other torch or Python
    may load it.  Written beside it."""
    return f"torch {torch_version} {sysconfig.get_config_var('SOABI')}"


def _torch_version(torch: str) -> str:
    return runpy.run_path(os.path.join(torch, "version.py"))["__version__"]


def _lib_newest() -> bool:
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime()


def _call_newest() -> bool:
    torch = _torch()
    if torch is None:
        return True
    try:
        with open(CALL_FOR) as f:
            made_for = f.read()
    except OSError:
        return False
    return (made_for == call_made_for(_torch_version(torch)) and os.path.exists(CALL) and
            os.path.getmtime(CALL) >= _deps_mtime())


def _newest() -> bool:
    return _lib_newest() and _call_newest()


def _build_call() -> None:
    """The tensor wrappers' common case, a CPython module of its own (torch's libraries are loaded before it is).  The
    wrappers go on without it, so what its compiler refuses is told and stops nothing."""
    tmp, torch = CALL + f".tmp{os.getpid()}", _torch()
    if torch is None:
        return
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(torch, "include"), "-isystem",
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
           os.path.join(CSRC, "tqd_call.cpp"), "-o", tmp, "-L", os.path.join(torch, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-ldl"]
    if os.path.exists(CALL_FOR):
        os.remove(CALL_FOR)  # (one from other sources is not loaded meanwhile, nor if this fails)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = r.stdout + r.stderr if r.returncode else None
    except OSError as e:
        why = str(e)
    if why is not None:
        warnings.warn(f"the call module was not built, calls with tensors are marshalled in Python: g++ failed for tqd_call.cpp:\n{why}",
                      RuntimeWarning)
        return
    os.replace(tmp, CALL)
    with open(CALL_FOR + f".tmp{os.getpid()}", "w") as f:
        f.write(call_made_for(_torch_version(torch)))
    os.replace(CALL_FOR + f".tmp{os.getpid()}", CALL_FOR)


def build(force: bool = False, verbose: bool = False, extra: list | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(1) as ex:
        call = ex.submit(_build_call) if force or not _call_newest() else None
        if force or not _lib_newest():
            _build_lib(verbose, extra)
        if call:
            call.result()
    return LIB


def _build_lib(verbose: bool, extra: list | None) -> None:
    extra = list(extra or [])
    if verbose:
        extra += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    def compile_synth():
        # the seeded input generator, linked in for tqd_create_synthetic (the
        # same source and flags as the Python synth module's own build)
        obj = os.path.join(BUILD, "tqd_synth.o")
        cmd = ["gcc", "-O2", "-std=c11", "-fPIC", "-fopenmp", "-ffp-contract=off", "-fno-fast-math", "-c",
               SYNTH_SRC, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"gcc failed for tqd_synth.c:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        futs = [ex.submit(compile_one, src) for src in SOURCES] + [ex.submit(compile_synth)]
        results = [f.result() for f in futs]
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart", "-lgomp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
