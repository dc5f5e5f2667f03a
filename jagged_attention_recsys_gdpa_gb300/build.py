"""Compile the CUDA library ``libjattn.so`` in-tree for sm_103a.

Each translation unit is compiled by its own nvcc process (in parallel),
then linked into ``_build/libjattn.so`` next to this file. The host calls of the
row operators and the page pool (``csrc/host.cpp``, on CPython's C API and
PyTorch's headers) become the extension module ``_build/_host.so``, which fits
the PyTorch and the Python that it was built for (``_build/_host.for``) and is built
again for others. Nothing is installed; the binding loads both from that path.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libjattn.so")
HOST = os.path.join(BUILD, "_host.so")
HOST_FOR = os.path.join(BUILD, "_host.for")
SOURCES = ["api.cu", "sched.cu", "fwd.cu", "fwd_block.cu", "fwd_hilo.cu", "fwd_block_hilo.cu", "bwd.cu",
           "bwd_hilo.cu", "fwd_mx.cu", "bwd_mx.cu", "pma.cu", "rope.cu", "mx.cu", "cache.cu", "decode.cu",
           "norm.cu", "norm_bwd.cu", "rotary.cu", "pages.cu", "partition.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "jattn.h"))
    return files


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _installed() -> str:
    """What _host.so depends on beside its sources."""
    import torch

    return f"PyTorch {torch.__version__} {torch.version.git_version}, Python {sysconfig.get_config_var('SOABI')}"


def host_misfit() -> str:
    """What _host.so was built for, where that is not what is installed, else nothing."""
    try:
        with open(HOST_FOR) as f:
            built = f.read()
    except FileNotFoundError:
        built = "an unknown PyTorch"
    return "" if built == _installed() else built


def _build_host() -> None:
    """The extension module, compiled against the PyTorch that is installed."""
    import torch

    root = os.path.dirname(torch.__file__)
    inc, libs = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    tmp = HOST + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
           os.path.join(CSRC, "host.cpp"), "-o", tmp, "-L", libs, f"-Wl,-rpath,{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on host.cpp:\n{r.stderr[-6000:]}")
    os.replace(tmp, HOST)
    with open(tmp, "w") as f:
        f.write(_installed())
    os.replace(tmp, HOST_FOR)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library's path. Where the extension module fails, the error comes after the library has been built: attention and
    the paged cache need nothing of it."""
    os.makedirs(BUILD, exist_ok=True)
    deps = _deps()
    library, host = force or _stale(LIB, deps), force or _stale(HOST, deps) or host_misfit() != ""
    with ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(_build_host) if host else None
        if library:
            _build_library()
    if module is not None:
        module.result()
    if verbose and library:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


def _build_library() -> None:
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-Xptxas", "-v", "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        with open(obj + ".log", "w") as f:
            f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr[-6000:]}")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
