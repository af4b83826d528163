"""In-tree build of the CUDA library ``libfa_gb300.so`` for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled by ``nvcc`` in parallel into
``_build/``, then linked into one shared library next to this file. Only one
``-gencode`` target is built (``compute_103a`` / ``sm_103a``). Rebuilds happen
when a source or header is newer than the library.

``csrc/fa_binding.cpp``, the marshalling of torch tensors for the packed and paged
calls, becomes the Python module ``_fa_binding.<abi>.so`` beside it, linked to the
library and built for the Python and the torch that are installed, which its name states:
with another torch it is not found, and build() makes that one's.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

import torch

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIBRARY = os.path.join(PKG_DIR, "libfa_gb300.so")
BINDING = os.path.join(
    PKG_DIR, f"_fa_binding.{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}.so")

SOURCES = ["fa_api.cu", "fa_forward.cu", "fa_backward.cu", "fa_softmax.cu", "fa_selftest.cu",
           "fa_noalloc.cu", "fa_session.cu", "fa_standard.cu", "fa_packed_plan.cu",
           "fa_packed_forward.cu", "fa_packed_backward.cu", "fa_packed_api.cu",
           "fa_cache.cu", "fa_prefix.cu", "fa_decode_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
             if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not (os.path.exists(LIBRARY) and os.path.exists(BINDING)):
        return False
    t = min(os.path.getmtime(LIBRARY), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library; returns its path."""
    if not force and up_to_date():
        return LIBRARY
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    def compile_binding():
        root = os.path.dirname(torch.__file__)  # its headers and libraries
        include = [os.path.join(root, "include"),
                   os.path.join(root, "include", "torch", "csrc", "api", "include"),
                   sysconfig.get_paths()["include"], INCLUDE]
        obj = os.path.join(BUILD_DIR, "fa_binding.o")
        r = subprocess.run([nvcc, "-O2", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                            *("-I" + p for p in include), "-c",
                            os.path.join(CSRC, "fa_binding.cpp"), "-o", obj],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"the compiler failed on fa_binding.cpp:\n{r.stdout}\n{r.stderr}")
        return obj, os.path.join(root, "lib")

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding_obj, torch_lib = binding.result()
    tmp = LIBRARY + f".tmp{os.getpid()}"
    # The name under which the binding asks for it, and finds it beside itself ($ORIGIN).
    r = subprocess.run([nvcc, *ARCH, "-shared", "-Xlinker",
                        "-soname=" + os.path.basename(LIBRARY), "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBRARY)
    tmp = BINDING + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, "-shared", "-cudart", "none", "-o", tmp, binding_obj, LIBRARY,
                        "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                        "-Xlinker", "-rpath=$ORIGIN"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return LIBRARY


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
