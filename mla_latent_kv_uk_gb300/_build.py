"""In-tree build of the CUDA library (sm_103a) with nvcc.

Compiles every ``csrc/*.cu`` to an object in parallel, then links
``_lib/libmla_gb300.so`` (static CUDA runtime, no driver-library link:
the TMA encoder is resolved through the runtime's driver entry points).
``csrc/binding.cpp``, the part of the Python binding that is compiled, becomes
``_lib/_mla_binding.so`` beside it: against the headers of the interpreter and
of the PyTorch that are there, and loaded by the package only.
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libmla_gb300.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"),
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def lib_path() -> str:
    return os.path.join(OUT_DIR, LIB_NAME)


def binding_path() -> str:
    return os.path.join(OUT_DIR, "_mla_binding.so")


def _build_binding(verbose: bool) -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch not found")
    torch = list(spec.submodule_search_locations)[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    libs = os.path.join(torch, "lib")
    tmp = binding_path() + ".tmp"
    cmd = [os.environ.get("CXX") or "g++", "-shared", "-fPIC", "-std=c++17", "-O2", "-o", tmp,
           os.path.join(CSRC, "binding.cpp"),
           *("-I" + d for d in (INCLUDE, os.path.join(torch, "include"),
                                os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                                sysconfig.get_paths()["include"], os.path.join(cuda, "include"))),
           "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, binding_path())


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_build_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = lib_path() + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path())
    binding.result()        # (the library is there whatever became of it)
    return lib_path()


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
