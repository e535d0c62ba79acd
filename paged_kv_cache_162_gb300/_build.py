"""Builds libpagedkv.so in-tree for sm_103a (nvcc, no cmake), and
_tensor_bind.so, which calls it with torch tensors (g++ against torch).

Each translation unit compiles in parallel; the link uses the shared CUDA
runtime so the library and PyTorch share one runtime in a process.

PKV_NVTX=1 in the environment builds the library with an NVTX range around
every C-ABI call (for profilers); the default build has none.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
BIND = os.path.join(PKG, "_tensor_bind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CU_SOURCES = ["runtime.cu", "cache_ops.cu", "decode.cu", "bounded.cu", "evict.cu"]
CXX_SOURCES = ["allocator.cpp", "beam_step.cpp"]
BIND_SOURCE = "tensor_bind.cpp"


def cuda_home() -> str:
    env = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if env and os.path.exists(os.path.join(env, "bin", "nvcc")):
        return env
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _nvcc() -> str:
    return os.path.join(cuda_home(), "bin", "nvcc")


def _inputs():
    """Every file the library is built from: all of csrc (sources and the
    headers they include), the public header and this script."""
    srcs = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
            if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    return srcs + [os.path.join(INCLUDE, "pagedkv.h"), os.path.abspath(__file__)]


FLAGS = os.path.join(BUILD, "flags.txt")


def _defines() -> list[str]:
    return ["-DPKV_NVTX"] if os.environ.get("PKV_NVTX", "") not in ("", "0") else []


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BIND):
        return False
    built = open(FLAGS).read() if os.path.exists(FLAGS) else ""
    if built != " ".join(_defines()):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _torch_flags():
    """(compile, link) flags against the torch that will load the module."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(root, "lib")
    return ([f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             *[x for p in inc for x in ("-isystem", p)]],
            ["-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"])


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    inc = ["-I", INCLUDE, "-I", CSRC]
    if os.path.basename(src) == BIND_SOURCE:
        inc += _torch_flags()[0]
    if src.endswith(".cu"):
        cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
               "-Xptxas", "-warn-spills", *inc, *extra, "-c", src, "-o", obj]
    else:
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra", *inc,
               *[x for x in extra if x.startswith("-D")],
               "-I", os.path.join(cuda_home(), "include"), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = (["-Xptxas", "-v"] if verbose_ptxas else []) + _defines()
    srcs = [os.path.join(CSRC, s) for s in [BIND_SOURCE] + CU_SOURCES + CXX_SOURCES]
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    bind, objs = objs[0], objs[1:]
    libdir = os.path.join(cuda_home(), "lib64")
    for out, cmd in (
            (LIB, [_nvcc(), *ARCH, "-shared", "-cudart", "shared", *objs,
                   "-Xlinker", f"-rpath,{libdir}"]),
            (BIND, ["g++", "-shared", bind, "-L", PKG, "-l:libpagedkv.so", "-Wl,-rpath,$ORIGIN",
                    *_torch_flags()[1]])):
        tmp = out + f".tmp{os.getpid()}"
        cmd = [*cmd, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, out)
    with open(FLAGS, "w") as f:
        f.write(" ".join(_defines()))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
