"""Build libmttkrp.so in-tree with nvcc for sm_103a (GB300), and the Python
module _binding.so with the host compiler.

Every source under csrc/ is compiled in parallel into _build/, then the .cu
files are linked into a shared library next to this file, and binding.cpp,
which calls that library, into a module next to it.  Rebuilds only when a
source or header is newer than what it goes into; the module also when it was
built for another Python or PyTorch.  Without PyTorch there is only the library.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmttkrp.so")
BINDING = os.path.join(HERE, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-Wall", f"-I{INCLUDE}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA 13 toolkit required)")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _binding_source():
    return os.path.join(CSRC, "binding.cpp")


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h"))) + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [os.path.join(INCLUDE, "mttkrp.h")]


def _newer(built: str, sources) -> bool:
    """Whether `built` exists and no source is newer."""
    return os.path.exists(built) and all(os.path.getmtime(p) <= os.path.getmtime(built) for p in sources)


def _fits() -> str | None:
    """The Python and PyTorch that a binding built now fits; None without PyTorch."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:     # not installed as a package
        import torch
        version = torch.__version__
    return f"{sys.implementation.cache_tag} {sysconfig.get_platform()} torch {version}"


def _fits_file() -> str:
    return os.path.join(BUILD, "binding.fits")


def _library_up_to_date() -> bool:
    return _newer(LIB, _sources() + _headers())


def _binding_up_to_date() -> bool:
    fits = _fits()
    if fits is None:
        return True                 # cannot be built
    if not _newer(BINDING, [_binding_source()] + _headers()) or not os.path.exists(_fits_file()):
        return False
    with open(_fits_file()) as f:
        return f.read() == fits


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def _torch_flags():
    """Flags to compile and link against the installed PyTorch and CUDA runtime headers."""
    import torch
    home = os.path.dirname(torch.__file__)
    include = os.path.join(home, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    flags = [f"-I{INCLUDE}", f"-I{sysconfig.get_paths()['include']}", "-isystem", include, "-isystem",
             os.path.join(include, "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    links = [f"-L{os.path.join(home, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return flags, links


def _run(cmd, what):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stderr}")
    return res


def build(force: bool = False, verbose: bool = False) -> str:
    library, fits = force or not _library_up_to_date(), _fits()
    module = fits is not None and (force or not _binding_up_to_date())
    if not library and not module:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags, links = _torch_flags() if module else ([], [])

    def compile_one(src):
        name = os.path.basename(src)
        obj = os.path.join(BUILD, os.path.splitext(name)[0] + ".o")
        if src.endswith(".cu"):
            cmd = [cc] + NVCC_FLAGS + ["-c", src, "-o", obj]
        else:
            cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall"] + flags + ["-c", src, "-o", obj]
        res = _run(cmd, f"compiling {src}")
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    srcs = ([_binding_source()] if module else []) + (_sources() if library else [])
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    binding = objs.pop(0) if module else None
    if library:
        tmp = LIB + f".tmp{os.getpid()}"
        _run([cc] + ARCH + ["-shared", "-o", tmp] + objs, "linking the library")
        os.replace(tmp, LIB)
    if module:
        tmp = BINDING + f".tmp{os.getpid()}"
        _run(["g++", "-shared", "-o", tmp, binding, f"-L{HERE}", "-lmttkrp", "-Wl,-rpath,$ORIGIN"] + links,
             "linking the binding")
        os.replace(tmp, BINDING)
        with open(_fits_file(), "w") as f:
            f.write(fits)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
