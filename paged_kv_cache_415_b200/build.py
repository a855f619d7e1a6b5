"""Build libpa.so (the C-ABI CUDA library) and _marshal.so (the torch side of
the calls that take strided tensors) in place, for sm_100a.

    python -m paged_kv_cache_415_b200.build [--force]

Each .cu file under csrc/ is compiled by nvcc in parallel
(-gencode arch=compute_100a,code=sm_100a -O3 -lineinfo, no fast-math) and
linked with the static CUDA runtime into paged_kv_cache_415_b200/libpa.so.
csrc_py/marshal.cpp is compiled by g++ against torch's headers.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libpa.so")
MARSHAL_SOURCE = os.path.join(HERE, "csrc_py", "marshal.cpp")
MARSHAL = os.path.join(HERE, "_marshal.so")
BUILD_DIR = os.path.join(ROOT, "_build")
MARSHAL_KEY = os.path.join(BUILD_DIR, "_marshal.key")      # what _marshal.so was built for

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-I" + INCLUDE, "-I" + CSRC,
]


def _nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _newer(target, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps)


def _read(path) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def build_marshal(force: bool = False) -> str:
    """_marshal.so, a CPython extension over torch's tensors.  Built anew as
    well when Python or torch is another one than it was built for."""
    import torch
    built_for = f"{sys.implementation.cache_tag} torch {torch.__version__}"
    deps = [MARSHAL_SOURCE, os.path.join(INCLUDE, "pa.h"), os.path.abspath(__file__)]
    if not force and _newer(MARSHAL, deps) and _read(MARSHAL_KEY) == built_for:
        return MARSHAL
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    root = os.path.dirname(torch.__file__)
    lib, inc = os.path.join(root, "lib"), os.path.join(root, "include")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f'-DPA_TORCH_VERSION="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + INCLUDE, "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
           "-isystem" + inc, "-isystem" + os.path.join(inc, "torch", "csrc", "api", "include"),
           MARSHAL_SOURCE, "-o", tmp, "-L" + lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on {MARSHAL_SOURCE}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, MARSHAL)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(MARSHAL_KEY, "w") as f:
        f.write(built_for)
    return MARSHAL


def build(force: bool = False, verbose: bool = False) -> str:
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        marshal = ex.submit(build_marshal, force)
        lib = _build_library(force, verbose)
        marshal.result()
    return lib


def _build_library(force: bool, verbose: bool) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        return obj, res.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static",
           "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
