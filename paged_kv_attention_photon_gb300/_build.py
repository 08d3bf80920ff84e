"""Build libphoton_paged.so in-tree with nvcc for sm_103a (GB300), and the Python
module _binding beside it.

One object per translation unit, compiled in parallel, then linked into a
shared library next to this file.  Rebuilds only when a source is newer than
the library.  No cmake, no torch extension machinery.

The library needs nvcc alone.  The module needs Python's headers too and carries
the tag of the Python it was built for; without the headers it is left out, and
only the calls that go through it raise.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
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
LIB_NAME = "libphoton_paged.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
BINDING_SRC = os.path.join(CSRC, "python", "binding.cpp")
BINDING_PATH = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--threads", "1", "-I" + INCLUDE]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libphoton_paged.so")


def sources() -> List[str]:
    """CUDA translation units and the plain host C++ ones (compiled by nvcc too,
    which hands .cpp files to the host compiler)."""
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _newer(path: str, deps: List[str]) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def _headers() -> List[str]:
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _python_include() -> Optional[str]:
    """The directory of Python.h, or None where it is not installed."""
    path = sysconfig.get_paths()["include"]
    return path if os.path.exists(os.path.join(path, "Python.h")) else None


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def binding_up_to_date() -> bool:
    return _newer(BINDING_PATH, [BINDING_SRC] + _headers())


def up_to_date() -> bool:
    return library_up_to_date() and (binding_up_to_date() or _python_include() is None)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          extra_flags: Optional[List[str]] = None) -> str:
    if not force and up_to_date():
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = ARCH_FLAGS + NVCC_FLAGS + list(extra_flags or [])
    if ptxas_info:
        flags = flags + ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    def link(objs: List[str]) -> None:
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc] + ARCH_FLAGS + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)

    def build_binding() -> None:
        if os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)   # of older declarations
        include = _python_include()
        if include is None:
            sys.stderr.write("Python.h is not installed: built without the Python module _binding\n")
            return
        tmp = BINDING_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I" + INCLUDE,
               "-I" + include, "-o", tmp, BINDING_SRC]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"the Python module failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BINDING_PATH)

    with cf.ThreadPoolExecutor(max_workers=max(2, min(len(sources()) + 1, os.cpu_count() or 4))) as ex:
        binding = None if not force and binding_up_to_date() else ex.submit(build_binding)
        if force or not library_up_to_date():
            link(list(ex.map(compile_one, sources())))
        if binding is not None:
            binding.result()
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
