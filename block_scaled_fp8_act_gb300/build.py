"""Build libfp8act.so in-tree with nvcc for sm_103a (GB300).

Each .cu file under csrc/ compiles to an object in parallel, then nvcc links
the shared library against the shared CUDA runtime (the same libcudart.so.13
PyTorch loads). csrc/binding.cpp, the Python binding of the operators between
the linear layers, compiles with the host compiler against PyTorch's headers
into an extension module beside it, linked to the library; without PyTorch only
the library is built, for callers of the C ABI. No CMake; a rebuild happens only
when a source is newer than the libraries.
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
LIB_PATH = os.path.join(BUILD_DIR, "libfp8act.so")
INCLUDE = os.path.join(ROOT, "include")
BINDING = os.path.join(CSRC, "binding.cpp")
EXT_PATH = os.path.join(BUILD_DIR, "_fp8act.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfp8act")
    return path


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + [BINDING] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _stale() -> bool:
    made = [LIB_PATH, EXT_PATH] if _has_torch() else [LIB_PATH]
    if not all(os.path.exists(p) for p in made):
        return True
    t = min(os.path.getmtime(p) for p in made)
    return any(os.path.getmtime(p) > t for p in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every CUDA source and link libfp8act.so, and the binding; returns the library's path."""
    if not force and not _stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose or ptxas_info:
            print(r.stderr, end="")
        return obj

    def run(cmd: list[str], what: str) -> None:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stderr}")

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding, cc, run) if _has_torch() else None
        objs = list(ex.map(compile_one, sources()))
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        run([cc, *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp,
             "-Xlinker", "-rpath", "-Xlinker", "/usr/local/cuda/lib64"], "nvcc link")
        os.replace(tmp, LIB_PATH)
        if binding:
            _link_binding(cc, run, binding.result())
    return LIB_PATH


def _cuda_dir(cc: str) -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(cc)))


def _compile_binding(cc: str, run) -> str:
    import torch

    torch_dir = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD_DIR, "binding.cpp.o")
    run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-I", os.path.join(torch_dir, "include"), "-I", sysconfig.get_paths()["include"],
         "-I", os.path.join(_cuda_dir(cc), "include"), "-c", BINDING, "-o", obj], f"g++ on {BINDING}")
    return obj


def _link_binding(cc: str, run, obj: str) -> None:
    import torch

    tmp = EXT_PATH + f".tmp{os.getpid()}"
    torch_lib, cuda_lib = os.path.join(os.path.dirname(torch.__file__), "lib"), os.path.join(_cuda_dir(cc), "lib64")
    run(["g++", "-shared", obj, "-o", tmp, "-L", BUILD_DIR, "-l:libfp8act.so", "-L", torch_lib, "-ltorch_python",
         "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", cuda_lib, "-lcudart",
         f"-Wl,-rpath,$ORIGIN,-rpath,{torch_lib},-rpath,{cuda_lib}"], "linking the binding")
    os.replace(tmp, EXT_PATH)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
