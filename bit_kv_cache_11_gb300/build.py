"""Builds the in-tree CUDA library ``libkvq.so`` for sm_103a with nvcc.

Every ``csrc/*.cu`` file is compiled to an object in parallel, then linked
into one shared library (static CUDA runtime, C ABI of ``include/kvq.h``).
``csrc/paged_bind.cpp``, the Python binding of the paged cache's calls, is
compiled beside them against torch's headers into ``_paged_bind.so``.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkvq.so")
BIND = os.path.join(PKG, "_paged_bind.so")
CXX = os.environ.get("CXX", "g++")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_commands(obj: str, out: str) -> tuple[list, list]:
    """The commands that compile and link the Python binding."""
    import torch
    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), sysconfig.get_paths()["include"],
               os.path.join(CUDA, "include"), os.path.join(ROOT, "include")]
    lib = os.path.join(root, "lib")
    return ([CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
             *(x for d in include for x in ("-I", d)),
             "-c", os.path.join(CSRC, "paged_bind.cpp"), "-o", obj],
            [CXX, "-shared", "-o", out, obj, "-L" + PKG, "-l:libkvq.so", "-L" + lib, "-lc10",
             "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
             "-L" + os.path.join(CUDA, "lib64"), "-lcudart",
             "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile and link libkvq.so if any source changed; returns its path."""
    os.makedirs(OBJ, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(ROOT, "include", "kvq.h")]
    objs = []
    todo = []
    for src in sources:
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, *headers]):
            todo.append((src, obj))

    bind_obj = os.path.join(OBJ, "paged_bind.o")
    bind_src = os.path.join(CSRC, "paged_bind.cpp")
    bind = _bind_commands(bind_obj, BIND + f".tmp{os.getpid()}")
    if force or _stale(bind_obj, [bind_src, os.path.join(ROOT, "include", "kvq.h")]):
        todo.insert(0, (bind_src, bind_obj))

    def compile_one(job):
        src, obj = job
        cmd = bind[0] if obj == bind_obj else [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on {src}:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    if todo:
        with ThreadPoolExecutor(max_workers=jobs or min(len(todo), os.cpu_count() or 4)) as ex:
            for msg in ex.map(compile_one, todo):
                if verbose and msg:
                    print(msg)
    if force or todo or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if force or todo or _stale(BIND, [bind_obj]):
        r = subprocess.run(bind[1], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(BIND + f".tmp{os.getpid()}", BIND)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
