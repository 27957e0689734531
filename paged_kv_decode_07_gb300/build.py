"""Builds libpa.so (the C ABI of include/pa.h) in-tree with nvcc for sm_103a,
and the Python extension _pa_py.so (csrc/pa_py.cpp) with the host compiler.

Each .cu in csrc/ compiles to an object in parallel; the objects link into
paged_kv_decode_07_gb300/libpa.so with the CUDA runtime linked statically,
so the library loads without a separate libcudart on the path.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(ROOT, "_build", "pa")
LIB = os.path.join(HERE, "libpa.so")
EXT = os.path.join(HERE, "_pa_py.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "pa.h"))
    return max(os.path.getmtime(f) for f in files)


def up_to_date() -> bool:
    return all(os.path.exists(f) and os.path.getmtime(f) >= _deps_mtime() for f in (LIB, EXT))


def _compile_ext() -> None:
    """The extension uses torch's tensors: compiled against the installed torch."""
    import torch

    base = torch.__path__[0]
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++20", "-fPIC", "-shared", "-w", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           os.path.join(CSRC, "pa_py.cpp"), "-o", tmp, "-L", os.path.join(base, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for pa_py.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        ext = ex.submit(_compile_ext)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        ext.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
