"""Build libgemm07.so in-tree with nvcc for sm_103a (no CMake, no setuptools),
and the torch binding of the layer operators beside it.

Each ``csrc/*.cu`` translation unit is compiled in parallel to an object
under ``_build/`` and the objects are linked into ``_lib/libgemm07.so``
(CUDA runtime linked statically).  ``csrc/layer_binding.cpp`` is compiled with
the host compiler against the installed torch into ``_lib/layer_binding.so``,
which is linked to the library.  A rebuild happens only when a source or
header is newer than the libraries.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libgemm07.so")
BINDING_SRC = os.path.join(CSRC, "layer_binding.cpp")
BINDING_PATH = os.path.join(LIB_DIR, "layer_binding.so")
HEADER = os.path.join(ROOT, "include", "gemm07.h")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = [os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc"),
            shutil.which("nvcc") or ""]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found (set CUDA_HOME)")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [BINDING_SRC, HEADER, __file__]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _host(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _compile_binding() -> str:
    obj = os.path.join(BUILD_DIR, "layer_binding.o")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(_torch_dir(), "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    _host(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"] + [f"-I{d}" for d in inc] +
          ["-c", BINDING_SRC, "-o", obj], "g++ on layer_binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    libs = os.path.join(_torch_dir(), "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    _host(["g++", "-shared", "-o", tmp, obj, f"-L{LIB_DIR}", "-lgemm07", f"-L{libs}", "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN",
           f"-Wl,-rpath,{libs}"], "linking layer_binding.so")
    os.replace(tmp, BINDING_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    srcs = sources()
    workers = max(1, min(len(srcs) + 1, os.cpu_count() or 4))
    with ThreadPoolExecutor(max_workers=workers) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(compile_one, srcs))
        binding_obj = binding.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_binding(binding_obj)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
