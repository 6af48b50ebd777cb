"""Builds libembbwd.so in-tree: every csrc/*.cu compiled for sm_103a in parallel, then linked;
and, where there is a PyTorch with CUDA, _vocab.so, the Python entry of the vocabulary operators
(csrc/vocab_torch.cpp), beside it.

    python -m sparse_embedding_bag_gb300.build [--force] [--ptxas-v]
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libembbwd.so")
ENTRY_SRC = os.path.join(CSRC, "vocab_torch.cpp")
ENTRY = os.path.join(PKG, "_vocab.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def build_entry() -> None:
    """_vocab.so: host code against this machine's PyTorch headers (no link to libembbwd: it is
    given the functions' addresses when it is loaded). The library itself does without PyTorch."""
    import sysconfig

    if not has_torch():
        return
    import torch
    from torch.utils import cpp_extension
    if torch.version.cuda is None:
        return
    include = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = ENTRY + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(x for p in include for x in ("-isystem", p)), ENTRY_SRC, "-o", tmp, "-L" + lib, "-Wl,-rpath," + lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {ENTRY_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, ENTRY)


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int | None = None) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    newest = _newest(deps + [ENTRY_SRC, __file__])
    made = (LIB, ENTRY) if has_torch() else (LIB,)
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= newest for p in made):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    jobs = jobs or min(len(srcs), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(jobs + 1) as ex:
        entry = ex.submit(build_entry)
        results = list(ex.map(compile_one, srcs))
        entry.result()
    if ptxas_verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_verbose="--ptxas-v" in sys.argv))
