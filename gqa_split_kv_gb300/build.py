"""Builds libdecode_attn.so in-tree with nvcc for sm_103a, and the binding's CPython extension with the host compiler
(no CMake; the units compile side by side).  The library needs nvcc and its host compiler alone; the extension needs the
headers of Python and of an installed PyTorch, and is left out where there are none."""
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
EXT_STAMP = os.path.join(PKG, "_build", "binding_ext.torch")  # the PyTorch that EXT was compiled against
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


def torch_dir():
    """The installed PyTorch's folder, or None (found without importing it)."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def torch_tag():
    """What tells one installed PyTorch from another."""
    torch = torch_dir()
    version = os.path.join(torch, "version.py")
    return torch + "\n" + (open(version).read() if os.path.exists(version) else "")


def ext_needs():
    """Why the extension cannot be built here, or None."""
    torch = torch_dir()
    if torch is None:
        return "PyTorch is not installed"
    for header in (os.path.join(torch, "include", "ATen", "core", "Tensor.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return "no " + header
    return None


def ext_command(out: str) -> list:
    """Compiles the binding's extension against the installed PyTorch."""
    torch = torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(torch, "lib")
    return [os.environ.get("CXX", "g++"), "-shared", "-fPIC", "-std=c++17", "-O2", *("-I" + i for i in include),
            EXT_SOURCE, "-o", out, "-L" + lib, "-Wl,-rpath," + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python", "-ldl"]


def _newer(out, sources) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in sources)


def library_up_to_date() -> bool:
    return _newer(LIB, SOURCES + HEADERS)


def ext_up_to_date() -> bool:
    return (_newer(EXT, [EXT_SOURCE, HEADERS[0]]) and os.path.exists(EXT_STAMP) and
            open(EXT_STAMP).read() == torch_tag())


def _run(cmd: list):
    return subprocess.run(cmd, capture_output=True, text=True)


def _install(made: str, out: str):
    shutil.copy(made, out + ".tmp")
    os.replace(out + ".tmp", out)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is older than its sources: the library, and the extension where it can be built (compiled against
    another PyTorch counts as old).  Returns the library's path; a failing extension leaves the library in place."""
    missing = ext_needs()
    want_lib = force or not library_up_to_date()
    want_ext = missing is None and (force or not ext_up_to_date())
    if missing is not None:
        print(f"the binding's extension is not built: {missing}")
    if not want_lib and not want_ext:
        return LIB

    def report(res):
        if verbose or res.returncode != 0:
            print(" ".join(res.args))
            print(res.stdout + res.stderr)
        return res.returncode == 0

    with tempfile.TemporaryDirectory() as tmpdir:
        objects = [os.path.join(tmpdir, os.path.basename(src) + ".o") for src in SOURCES] if want_lib else []
        ext = os.path.join(tmpdir, "ext.so")
        with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as pool:
            ext_job = pool.submit(_run, ext_command(ext)) if want_ext else None
            jobs = [pool.submit(_run, nvcc_command(out, src)) for out, src in zip(objects, SOURCES)]
        if want_lib:
            lib = os.path.join(tmpdir, "lib.so")
            if not all([report(job.result()) for job in jobs]) or not report(_run(link_command(lib, objects))):
                raise RuntimeError("nvcc failed building libdecode_attn.so")
            _install(lib, LIB)
        if ext_job:
            if not report(ext_job.result()):
                raise RuntimeError("the host compiler failed building the binding's extension")
            _install(ext, EXT)
            os.makedirs(os.path.dirname(EXT_STAMP), exist_ok=True)
            with open(EXT_STAMP, "w") as f:
                f.write(torch_tag())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
