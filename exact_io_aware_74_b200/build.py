"""Builds libfa2.so (the C-ABI CUDA library) in-tree for sm_100a.

    python -m exact_io_aware_74_b200.build [--force]

The library is written next to this file so that it travels with the source tree.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfa2.so")
BUILD = os.path.join(HERE, "_build")  # object files
SOURCES = [os.path.join(CSRC, f) for f in (
    "fa2_api.cu", "fa2_seq_api.cu", "fa2_seq_packed.cu", "fa2_seq_paged.cu",
    "fa2_seq_bwd.cu")]
HEADERS = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
    os.path.join(ROOT, "include", "fa2.h")]
DEPS = SOURCES + HEADERS

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in DEPS)


def _compile(src: str) -> tuple[str, str, int]:
    """One source to its object file, if that is older than the source or a header."""
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    log = obj + ".log"
    deps = [src, os.path.abspath(__file__), *HEADERS]
    if os.path.exists(obj) and os.path.exists(log) and all(
            os.path.getmtime(p) <= os.path.getmtime(obj) for p in deps):
        return obj, open(log).read(), 0
    tmp = obj + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    text = " ".join(cmd) + "\n" + res.stdout + res.stderr
    if res.returncode == 0:
        os.replace(tmp, obj)
        with open(log, "w") as f:
            f.write(text)
    return obj, text, res.returncode


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in os.listdir(BUILD):
            os.remove(os.path.join(BUILD, f))
    with ThreadPoolExecutor(len(SOURCES)) as pool:
        done = list(pool.map(_compile, SOURCES))
    text, rc = "".join(d[1] for d in done), max(d[2] for d in done)
    tmp = LIB + f".tmp{os.getpid()}"
    if rc == 0:
        cmd = [nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
               *(d[0] for d in done), "-o", tmp, "-lcuda"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        text, rc = text + " ".join(cmd) + "\n" + res.stdout + res.stderr, res.returncode
    log = os.path.join(HERE, "build.log")
    with open(log, "w") as f:
        f.write(text)
    if rc != 0:
        sys.stderr.write(text)
        raise RuntimeError(f"nvcc failed (exit {rc}); see {log}")
    os.replace(tmp, LIB)
    if verbose:
        sys.stdout.write(text)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
