"""Builds libpagedkv.so in-tree for sm_103a (nvcc, no cmake), and
_tensor_bind.so, which calls it with torch tensors (g++ against torch).  The
library needs no torch: without one, or where the module does not compile
against it, the library is built all the same and engine.py calls it through
ctypes.

Each translation unit compiles in parallel; the link uses the shared CUDA
runtime so the library and PyTorch share one runtime in a process.

PKV_NVTX=1 in the environment builds the library with an NVTX range around
every C-ABI call (for profilers); the default build has none.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
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
CU_SOURCES = ["runtime.cu", "cache_ops.cu", "decode.cu", "bounded.cu", "evict.cu", "rotary.cu", "q4_decode.cu"]
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
BIND_FLAGS = os.path.join(BUILD, "bind_flags.txt")


def _defines() -> list[str]:
    return ["-DPKV_NVTX"] if os.environ.get("PKV_NVTX", "") not in ("", "0") else []


def _torch_version() -> str:
    """The installed torch's version, without importing it; "" without one."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return ""
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        found = re.search(r"^__version__ = '([^']+)'", f.read(), re.M)
    return found.group(1) if found else ""


def _current(out: str, flags: str, want: str) -> bool:
    """`out` was built with the flags `want`, after the last change of any source."""
    if not os.path.exists(out) or not os.path.exists(flags):
        return False
    with open(flags) as f:
        if f.read() != want:
            return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _lib_current() -> bool:
    return _current(LIB, FLAGS, " ".join(_defines()))


def _bind_current() -> bool:
    torch = _torch_version()
    return not torch or _current(BIND, BIND_FLAGS, torch)


def up_to_date() -> bool:
    return _lib_current() and _bind_current()


def _torch_flags():
    """(compile, link) flags against the torch that will load the module."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(root, "lib")
    return ([f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             f'-DPKV_TORCH_VERSION="{torch.__version__}"',
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


def _link(out: str, cmd: list[str]) -> None:
    tmp = out + f".tmp{os.getpid()}"
    cmd = [*cmd, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _no_bind(error: Exception) -> None:
    """Says why there is no _tensor_bind.so; one of another build would not do."""
    if os.path.exists(BIND):
        os.remove(BIND)
    sys.stderr.write(f"_tensor_bind.so was not built; calls go through ctypes: {error}\n")


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    lib, bind = force or not _lib_current(), force or not _bind_current()
    if not lib and not bind:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = (["-Xptxas", "-v"] if verbose_ptxas else []) + _defines()
    srcs = [os.path.join(CSRC, s) for s in CU_SOURCES + CXX_SOURCES] if lib else []
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        bind_obj = ex.submit(_compile, os.path.join(CSRC, BIND_SOURCE), extra) if bind and _torch_version() else None
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    if lib:
        libdir = os.path.join(cuda_home(), "lib64")
        _link(LIB, [_nvcc(), *ARCH, "-shared", "-cudart", "shared", *objs, "-Xlinker", f"-rpath,{libdir}"])
        with open(FLAGS, "w") as f:
            f.write(" ".join(_defines()))
    if bind_obj is not None:
        try:
            _link(BIND, ["g++", "-shared", bind_obj.result(), "-L", PKG, "-l:libpagedkv.so", "-Wl,-rpath,$ORIGIN",
                         *_torch_flags()[1]])
        except Exception as e:  # whatever torch, its headers or g++ make of it
            _no_bind(e)
        else:
            with open(BIND_FLAGS, "w") as f:
                f.write(_torch_version())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
