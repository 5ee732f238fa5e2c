"""Build librkv.so in-tree for sm_103a with nvcc (translation units compiled in parallel),
and _pages.so, the Python binding of its page and prompt entry points, with the host compiler.

Usage: python -m residual_kv_cache_gb300.build   (or build() from Python)
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import platform
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "librkv.so")
EXT = os.path.join(HERE, "_pages.so")
EXT_SOURCE = "pages_torch.cpp"
SOURCES = ["rkv_api.cu", "k_elementwise.cu", "k_gemm.cu", "k_retrieve.cu", "k_reconstruct.cu",
           "k_noalloc.cu", "k_attention.cu", "k_pages.cu", "k_page_attention.cu", "k_prompt.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [_nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    log = os.path.join(BUILD, os.path.splitext(src)[0] + ".ptxas.txt")
    with open(log, "w") as f:
        f.write(r.stderr)
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _compile_ext() -> str:
    """Object of the Python binding: host code against this torch's and Python's headers."""
    import sysconfig

    import torch
    obj = os.path.join(BUILD, os.path.splitext(EXT_SOURCE)[0] + ".o")
    include = [os.path.join(os.path.dirname(torch.__file__), "include"), sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]
    cmd = ["g++", "-O2", "-fPIC", "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{p}" for p in include), "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SOURCE}:\n{r.stderr}")
    return obj


def _link(cmd, out: str):
    tmp = out + ".tmp"
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(out)} failed:\n{r.stderr}")
    os.replace(tmp, out)


def _stamp() -> str:
    """Machine, torch version and hash of every source and of this script: a library built on
    another architecture, against another torch or from other sources is rebuilt."""
    import torch
    h = hashlib.sha1(f"{platform.machine()} {torch.__version__} {sys.version}".encode())
    paths = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                   if f.endswith((".cu", ".cuh", ".h", ".cpp")))
    paths += [os.path.join(HERE, "..", "include", "rkv.h"), os.path.abspath(__file__)]
    for p in paths:
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile every translation unit for sm_103a and link librkv.so and _pages.so; returns
    librkv.so's path."""
    os.makedirs(BUILD, exist_ok=True)
    stamp_file = os.path.join(BUILD, "stamp")
    stamp = _stamp()
    if not force and os.path.exists(LIB) and os.path.exists(EXT) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read().strip() == stamp:
                return LIB
    import torch
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(_compile_ext)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        ext_obj = ext.result()
    _link([_nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs], LIB)
    _link(["g++", "-shared", ext_obj, f"-L{HERE}", "-l:librkv.so", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
           "-ltorch_cuda", "-lc10", "-lc10_cuda"], EXT)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force=True))
