"""Build libzs.so from csrc/*.cu with nvcc for sm_103a (GB300), and zs_torch,
the binding's short way from torch tensors to it, from csrc/zs_torch.cpp.  libzs
needs nvcc alone; zs_torch is of one torch and one Python, whose versions its
file is named by, and where it cannot be built the binding does without.

Each translation unit compiles in its own process, in parallel, then one link
step produces ``_build/libzs.so`` inside the package.  No GPU is needed to
build.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libzs.so")
EXT_SOURCE = os.path.join(CSRC, "zs_torch.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libzs needs the CUDA toolkit to build")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(target: str, deps: list[str]) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps + [__file__])


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr:
        sys.stderr.write(res.stderr)
    return obj


def ext_path() -> str:
    """Where zs_torch of the torch and Python that run this lies."""
    import torch

    return os.path.join(BUILD, f"zs_torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_ext(force: bool = False) -> str:
    """Compile zs_torch against the torch and Python that run this, unless it is up to date; returns its path."""
    path = ext_path()
    if not force and _newer(path, [EXT_SOURCE] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return path
    import torch
    from torch.utils import cpp_extension

    os.makedirs(BUILD, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    includes = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_paths()["include"], cuda]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = path + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-isystem{d}" for d in includes),
           EXT_SOURCE, "-o", tmp, f"-L{libs}", f"-Wl,-rpath,{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the build of zs_torch failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, path)
    return path


def _try_ext(force: bool) -> None:
    try:
        build_ext(force)
    except Exception as e:
        warnings.warn(f"zs_torch was not built, calls of the training operators take longer on the host: {e}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc/*.cu for sm_103a and link libzs.so (its path is returned), and zs_torch where that can be."""
    if not force and up_to_date():
        _try_ext(False)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        ext = ex.submit(_try_ext, force)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        ext.result()
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-lcudart_static"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of libzs.so failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
