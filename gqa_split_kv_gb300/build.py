"""Builds libdecode_attn.so in-tree with nvcc for sm_103a (no CMake; its units compile side by side)."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libdecode_attn.so")
SOURCES = [os.path.join(CSRC, f) for f in ("decode_attn.cu", "latent_attn.cu", "cache_ops.cu")]
HEADERS = [os.path.join(ROOT, "include", "decode_attn.h")] + [
    os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cuh", ".h"))
]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")


def nvcc_command(out: str, source: str, extra=()) -> list:
    """Compiles one unit to an object."""
    return [nvcc_path(), "-c", "-Xcompiler", "-fPIC", "-std=c++17", "-O3", "-lineinfo",
            "-gencode", "arch=compute_103a,code=sm_103a", *extra, "-o", out, source]


def link_command(out: str, objects) -> list:
    return [nvcc_path(), "-shared", "-Xcompiler", "-fPIC", "-gencode", "arch=compute_103a,code=sm_103a", "-o", out,
            *objects]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in SOURCES + HEADERS)


def _run(cmd: list):
    return subprocess.run(cmd, capture_output=True, text=True)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if any source is newer than it; returns its path."""
    if not force and up_to_date():
        return LIB
    with tempfile.TemporaryDirectory() as tmpdir:
        objects = [os.path.join(tmpdir, os.path.basename(src) + ".o") for src in SOURCES]
        with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
            done = list(pool.map(_run, map(nvcc_command, objects, SOURCES)))
        if all(res.returncode == 0 for res in done):
            tmp = LIB + ".tmp"
            done.append(_run(link_command(tmp, objects)))
    for res in done:
        if verbose or res.returncode != 0:
            print(" ".join(res.args))
            print(res.stdout + res.stderr)
    if any(res.returncode != 0 for res in done):
        raise RuntimeError("nvcc failed building libdecode_attn.so")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
