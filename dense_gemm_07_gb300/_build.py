"""Build libgemm07.so in-tree with nvcc for sm_103a (no CMake, no setuptools),
and the torch binding of the layer operators beside it.

Each ``csrc/*.cu`` translation unit is compiled in parallel to an object
under ``_build/`` and the objects are linked into ``_lib/libgemm07.so``
(CUDA runtime linked statically).  ``csrc/layer_binding.cpp`` is compiled with
the host compiler against the installed torch into ``_lib/layer_binding.so``,
which is linked to the library.  The library needs no torch, and is all that
the C entry points and the ctypes layer load.

A rebuild of either happens only when one of its sources or headers is newer,
and of the binding also when the installed torch or Python is another one than
it was compiled against (recorded under ``_build/``).
"""
from __future__ import annotations

import glob
import importlib.util
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
BINDING_STAMP = os.path.join(BUILD_DIR, "layer_binding.txt")  # what it was compiled against
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


def _newer(path, deps) -> bool:
    """path exists and is at least as new as all of deps."""
    return os.path.exists(path) and \
        all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _library_deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [HEADER, __file__]


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, _library_deps())


def _torch_dir() -> str | None:
    """Directory of a torch built for CUDA, or None; torch is not imported."""
    try:
        spec = importlib.util.find_spec("torch")
    except ValueError:
        return None
    if spec is None or not spec.origin:
        return None
    d = os.path.dirname(spec.origin)
    return d if os.path.exists(os.path.join(d, "lib", "libc10_cuda.so")) else None


def _torch_version(torch_dir: str) -> str:
    with open(os.path.join(torch_dir, "version.py")) as f:
        return f.read()


def _binding_stamp(torch_dir: str) -> str:
    return "\n".join([torch_dir, sysconfig.get_config_var("SOABI") or "",
                      _torch_version(torch_dir)])


def binding_up_to_date() -> bool:
    d = _torch_dir()
    if d is None or not _newer(BINDING_PATH, [BINDING_SRC, HEADER, __file__]):
        return False
    try:
        with open(BINDING_STAMP) as f:
            return f.read() == _binding_stamp(d)
    except FileNotFoundError:
        return False


def _run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")
    if verbose and r.stderr:
        print(r.stderr)


def _folders() -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and library_up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    _folders()

    def compile_one(src):
        name = os.path.basename(src)
        obj = os.path.join(BUILD_DIR, name[:-3] + ".o")
        _run([nvcc] + NVCC_FLAGS + ["-c", src, "-o", obj], f"nvcc on {name}", verbose)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    _run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs, "linking libgemm07.so")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _compile_binding(torch_dir: str) -> str:
    _folders()
    obj = os.path.join(BUILD_DIR, "layer_binding.o")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(torch_dir, "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"] + [f"-I{d}" for d in inc] +
         ["-c", BINDING_SRC, "-o", obj], "g++ on layer_binding.cpp")
    return obj


def _link_binding(torch_dir: str, obj: str) -> None:
    libs = os.path.join(torch_dir, "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{LIB_DIR}", "-lgemm07", f"-L{libs}", "-lc10",
          "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN",
          f"-Wl,-rpath,{libs}"], "linking layer_binding.so")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_stamp(torch_dir))


def build_binding(force: bool = False) -> str:
    """The binding (and the library that it is linked to)."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        raise RuntimeError("the layer operators need a torch built for CUDA")
    build_library()
    if force or not binding_up_to_date():
        _link_binding(torch_dir, _compile_binding(torch_dir))
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """The library and, where torch is installed, the binding."""
    torch_dir = _torch_dir()
    if torch_dir is None or not (force or not binding_up_to_date()):
        return build_library(force, verbose)
    with ThreadPoolExecutor(max_workers=1) as ex:  # beside the library's units
        obj = ex.submit(_compile_binding, torch_dir)
        build_library(force, verbose)
        _link_binding(torch_dir, obj.result())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
