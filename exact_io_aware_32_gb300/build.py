"""Builds the CUDA library libfa.so in-tree with nvcc, for sm_103a only.

Each translation unit is compiled in parallel; the objects are linked into
``exact_io_aware_32_gb300/_build/libfa.so`` with the CUDA runtime linked
statically, so the library has no dependency on libcuda at load time (the
driver's tensor-map encoder is looked up at run time).

``build_torch_module`` builds, with the host compiler, the small module through
which torch tensors reach the paged cache's calls: on its own, since the library
needs neither torch nor a host tool chain that can compile against it.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libfa.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_fwd_persist.cu", "fa_bwd.cu", "fa_bwd_noalloc.cu", "schedule.cu", "paged_api.cu",
           "paged_cache.cu", "paged_fwd.cu", "paged_few.cu", "paged_chunk.cu"]
HEADERS = ["ptx.cuh", "block_order.cuh", "fa_internal.h", "philox.cuh", "paged.h",
           "paged_work.cuh", "paged_pipe.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-diag-suppress", "177"]


def torch_module() -> str:
    """Path of the module built against the torch that is installed, for this interpreter (others are other files)."""
    import torch

    tags = (torch.__version__, sysconfig.get_config_var("SOABI") or sys.implementation.cache_tag)
    return os.path.join(BUILD, ".".join(["_fa_torch"] + [re.sub(r"[^0-9A-Za-z]+", "_", t) for t in tags] + ["so"]))


def _torch_module_cmd(out: str) -> list:
    import torch

    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    lib = os.path.join(root, "lib")
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [f"-I{i}" for i in inc] +
            [os.path.join(CSRC, "fa_torch.cpp"), "-o", out, f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python",
             "-ltorch_cpu", "-lc10_cuda", "-lc10"])


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa.so")
    return path


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "fa.h")]
    objs, procs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [s] + hdrs):
            cmd = [nvcc()] + ARCH + FLAGS + ["-c", s, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{out.decode(errors='replace')}")
        if verbose and out:
            sys.stderr.write(out.decode(errors="replace"))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout.decode(errors='replace')}")
        os.replace(tmp, LIB)
    return LIB


def build_torch_module(force: bool = False) -> str:
    path = torch_module()
    if force or _stale(path, [os.path.join(CSRC, "fa_torch.cpp")]):
        os.makedirs(BUILD, exist_ok=True)
        tmp = path + f".tmp{os.getpid()}"
        r = subprocess.run(_torch_module_cmd(tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on fa_torch.cpp:\n{r.stdout.decode(errors='replace')}")
        os.replace(tmp, path)
    return path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
