"""Builds the in-tree CUDA library ``libkvq.so`` for sm_103a with nvcc.

Every ``csrc/*.cu`` file is compiled to an object in parallel, then linked
into one shared library (static CUDA runtime, C ABI of ``include/kvq.h``).
``csrc/paged_bind.cpp``, the Python binding of the paged cache's calls, is
compiled beside them against torch's headers into ``_paged_bind.so``; without
torch the library is built alone.
"""
from __future__ import annotations

import glob
import importlib.util
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


def _run(cmd: list, verbose: bool = False) -> str:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _bind_commands(obj: str, out: str) -> tuple[list, list]:
    """The commands that compile and link the Python binding."""
    import torch
    root = os.path.dirname(torch.__file__)
    system = [os.path.join(root, "include"), sysconfig.get_paths()["include"],
              os.path.join(CUDA, "include")]
    lib = os.path.join(root, "lib")
    return ([CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
             "-I", os.path.join(ROOT, "include"), *(x for d in system for x in ("-isystem", d)),
             "-c", os.path.join(CSRC, "paged_bind.cpp"), "-o", obj],
            [CXX, "-shared", "-o", out, obj, "-L" + PKG, "-l:libkvq.so", "-L" + lib, "-lc10",
             "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
             "-L" + os.path.join(CUDA, "lib64"), "-lcudart",
             "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])


def _bind_stamp(commands: tuple) -> str:
    """What the binding's object depends on besides its sources: the commands, and
    the versions of torch and Python, whose C++ headers it is compiled against."""
    import torch
    return repr((commands, torch.__version__, sysconfig.get_config_var("SOABI")))


def _read(path: str) -> str | None:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile and link libkvq.so if any source changed, and the binding where
    torch is installed and its sources, its commands, torch or Python changed.
    Returns the library's path."""
    os.makedirs(OBJ, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    header = os.path.join(ROOT, "include", "kvq.h")
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [header]
    objs = []
    todo = []
    for src in sources:
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src, *headers]):
            todo.append([NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj])

    bind = None  # the binding's compile command, where it has to run
    if importlib.util.find_spec("torch") is not None:
        obj = os.path.join(OBJ, "paged_bind.o")
        compile_cmd, link_cmd = _bind_commands(obj, BIND)
        stamp, text = os.path.join(OBJ, "paged_bind.stamp"), _bind_stamp((compile_cmd, link_cmd))
        if (force or _read(stamp) != text or _stale(obj, [os.path.join(CSRC, "paged_bind.cpp"), header])
                or _stale(BIND, [obj])):
            bind = compile_cmd

    with ThreadPoolExecutor(max_workers=jobs or min(len(todo) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_run, bind, verbose) if bind else None
        for msg in ex.map(lambda cmd: _run(cmd, verbose), todo):
            if verbose and msg:
                print(msg)
        if todo or _stale(LIB, objs):
            tmp = LIB + f".tmp{os.getpid()}"
            _run([NVCC, *ARCH, "-shared", "-o", tmp, *objs])
            os.replace(tmp, LIB)
        if binding:
            msg = binding.result()
            if msg:
                print(msg)
            tmp = BIND + f".tmp{os.getpid()}"
            _run(_bind_commands(obj, tmp)[1])
            os.replace(tmp, BIND)
            with open(stamp, "w") as f:
                f.write(text)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
