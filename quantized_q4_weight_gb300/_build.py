"""Builds libqgemv.so in-tree with nvcc for sm_103a, and the Python binding
_binding.so with the host compiler.

Each translation unit compiles in its own process (in parallel), then nvcc
links the CUDA ones into one shared library with the CUDA runtime linked
statically, and the binding is linked against that library and torch.  A
build is skipped when both are newer than every source.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libqgemv.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(cand, "bin", "nvcc") if cand else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqgemv")
    return p


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")

    def compile_binding() -> str:
        from torch.utils import cpp_extension as ce
        obj = os.path.join(BUILD_DIR, "binding.o")
        inc = [f"-I{d}" for d in [*ce.include_paths(), sysconfig.get_paths()["include"],
                                  os.path.join(os.path.dirname(os.path.dirname(cc)), "include")]]
        run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", *inc, "-c", BINDING_SRC, "-o", obj],
            f"compiling {BINDING_SRC}")
        return obj

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, srcs))
        binding_obj = binding.result()
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    from torch.utils import cpp_extension as ce
    tmp = BINDING + ".tmp"
    dirs = [f"-L{d}" for d in ce.library_paths()] + [f"-Wl,-rpath,{d}" for d in ce.library_paths()]
    run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, binding_obj, f"-L{PKG}", "-lqgemv", "-Wl,-rpath,$ORIGIN",
         *dirs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], "linking the binding")
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
