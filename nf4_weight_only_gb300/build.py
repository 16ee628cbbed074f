"""Build libnf4.so (the CUDA kernels and the C ABI) in-tree for sm_103a with nvcc, and the binding's compiled
calls (csrc/nf4_python.c) with the host compiler, for the interpreter that runs this.  Where there is no C compiler or
no Python.h, the library is built without them: the binding then makes the same calls through ctypes."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from typing import List, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libnf4.so")
CALLS_PATH = os.path.join(BUILD_DIR, "nf4_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["nf4_api.cu", "nf4_quant.cu", "nf4_gemv.cu", "nf4_ring.cu", "nf4_kv.cu", "nf4_attn.cu",
           "nf4_rows.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs() -> List[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "nf4.h"))
    files.append(os.path.abspath(__file__))
    return files


def _calls_command(out: str) -> Optional[List[str]]:
    """What compiles the binding's calls, or None without a C compiler or Python's headers."""
    cc, include = shutil.which(os.environ.get("CC", "gcc")), sysconfig.get_paths()["include"]
    if cc is None or not os.path.exists(os.path.join(include, "Python.h")):
        return None
    return [cc, "-O2", "-shared", "-fPIC", "-I", include, os.path.join(CSRC, "nf4_python.c"), "-lm", "-o", out]


def is_stale() -> bool:
    built = [LIB_PATH] + ([CALLS_PATH] if _calls_command(CALLS_PATH) else [])
    if not all(os.path.exists(f) for f in built):
        return True
    t = min(os.path.getmtime(f) for f in built)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags: List[str] = ()) -> str:
    """Compile every source in parallel, then link the shared library.  Returns its path."""
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    procs, objs = [], []
    calls_tmp = CALLS_PATH + f".tmp{os.getpid()}"
    calls = _calls_command(calls_tmp)
    if calls:
        procs.append(("nf4_python.c",
                      subprocess.Popen(calls, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    else:
        print("no C compiler or no Python.h: the binding's compiled calls are left out", file=sys.stderr)
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out.strip() and (verbose or p.returncode != 0):
            print(out, file=sys.stderr)
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB_PATH)
    if calls:
        os.replace(calls_tmp, CALLS_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
