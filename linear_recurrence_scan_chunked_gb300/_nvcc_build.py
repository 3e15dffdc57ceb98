"""Build the CUDA library in-tree: csrc/*.cu -> _lib/liblrscan.so (sm_103a), and
the marshalling module csrc/binding.cpp -> _lib/_lrs_binding.so (host code on
PyTorch's headers, linked against the library).

Each translation unit is compiled in parallel, by nvcc or g++, then linked into
its shared object, the library with the CUDA runtime linked statically.
Rebuilds only when a source or header is newer than the objects, or PyTorch is
another version than they were built for.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "liblrscan.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(OUT_DIR, "_lrs_binding.so")
STAMP = os.path.join(OUT_DIR, "torch_version")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_flags():
    """Include and link flags of PyTorch's C++ headers (a plain extension module)."""
    import sysconfig
    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    lib = os.path.join(root, "lib")
    return ([f"-I{p}" for p in inc] + [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"],
            [f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"])


def _torch_version() -> str:
    import torch
    return torch.__version__


def _inputs():
    return [BINDING_SRC] + sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING) or not os.path.exists(STAMP):
        return False
    if open(STAMP).read() != _torch_version():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    tag = str(os.getpid())

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src) + f".{tag}.o")
        if src == BINDING_SRC:
            cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *torch_inc, "-c", src, "-o", obj]
        else:
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        log = os.path.join(OUT_DIR, os.path.basename(src) + ".ptxas.log")
        with open(log, "w") as f:
            f.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {src}:\n{r.stderr[-4000:]}")
        return obj

    torch_inc, torch_link = _torch_flags()
    bobj = os.path.join(OUT_DIR, os.path.basename(BINDING_SRC) + f".{tag}.o")
    btmp = BINDING + f".{tag}.tmp"
    objs = [os.path.join(OUT_DIR, os.path.basename(s) + f".{tag}.o") for s in sources()]
    tmp = LIB + f".{tag}.tmp"
    try:
        todo = [BINDING_SRC] + sources()
        with ThreadPoolExecutor(max(1, min(len(todo), os.cpu_count() or 1))) as ex:
            list(ex.map(compile_one, todo))
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
        os.replace(tmp, LIB)
        cmd = ["g++", "-shared", "-o", btmp, bobj, "-L", OUT_DIR, "-llrscan", "-Wl,-rpath,$ORIGIN", *torch_link]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
        os.replace(btmp, BINDING)
        with open(STAMP, "w") as f:
            f.write(_torch_version())
    finally:  # no objects or partial library left behind, whatever failed
        for f in objs + [tmp, bobj, btmp]:
            if os.path.exists(f):
                os.remove(f)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
