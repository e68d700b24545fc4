"""Builds libdecode_attn.so in-tree with nvcc for sm_103a, and the binding's CPython extension with the host compiler
(no CMake; the units compile side by side)."""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libdecode_attn.so")
SOURCES = [os.path.join(CSRC, f) for f in ("decode_attn.cu", "latent_attn.cu", "cache_ops.cu")]
EXT = os.path.join(PKG, "_binding_ext" + sysconfig.get_config_var("EXT_SUFFIX"))
EXT_SOURCE = os.path.join(CSRC, "binding_ext.cpp")
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


def ext_command(out: str) -> list:
    """Compiles the binding's extension against the installed PyTorch (found without importing it)."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(torch, "lib")
    return [os.environ.get("CXX", "g++"), "-shared", "-fPIC", "-std=c++17", "-O2", *("-I" + i for i in include),
            EXT_SOURCE, "-o", out, "-L" + lib, "-Wl,-rpath," + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python", "-ldl"]


def up_to_date() -> bool:
    def newer(out, sources):
        return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in sources)
    return newer(LIB, SOURCES + HEADERS) and newer(EXT, [EXT_SOURCE, HEADERS[0]])


def _run(cmd: list):
    return subprocess.run(cmd, capture_output=True, text=True)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if any source is newer than it; returns its path."""
    if not force and up_to_date():
        return LIB
    with tempfile.TemporaryDirectory() as tmpdir:
        objects = [os.path.join(tmpdir, os.path.basename(src) + ".o") for src in SOURCES]
        ext = os.path.join(tmpdir, "ext.so")
        commands = [*map(nvcc_command, objects, SOURCES), ext_command(ext)]
        with concurrent.futures.ThreadPoolExecutor(len(commands)) as pool:
            done = list(pool.map(_run, commands))
        if all(res.returncode == 0 for res in done):
            done.append(_run(link_command(os.path.join(tmpdir, "lib.so"), objects)))
        if all(res.returncode == 0 for res in done):
            for made, out in ((os.path.join(tmpdir, "lib.so"), LIB), (ext, EXT)):
                shutil.copy(made, out + ".tmp")
                os.replace(out + ".tmp", out)
    for res in done:
        if verbose or res.returncode != 0:
            print(" ".join(res.args))
            print(res.stdout + res.stderr)
    if any(res.returncode != 0 for res in done):
        raise RuntimeError("nvcc failed building libdecode_attn.so")
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
