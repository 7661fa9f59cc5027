"""Build libsegquant.so (the sm_100a kernels and the C ABI) in-tree with nvcc,
and its bounds-checked debug build libsegquant_debug.so (SQ_DEBUG_BOUNDS: every
plain global store of every kernel tests its index first; see
sq_debug_bounds_checks in include/segquant.h).

    python -m w8a8_gemm_b200.build [--force] [--debug]

The library is compiled for sm_100a only, without fast-math: the activation
and weight quantizers depend on IEEE round-to-nearest fp32 operations.  The CUDA
runtime is linked statically, so the library needs only the NVIDIA driver at
run time; driver entry points (tensor-map encoding) are resolved through the
runtime, so there is no link-time dependency on libcuda.

Beside it, _sqtorch.<interpreter>.<torch>.so: the short way from torch tensors to
the library's operators (csrc/torch_calls.cpp), compiled with the host compiler
against one Python and one torch, which its name tells.  It is optional: where it
cannot be built, or was built for others, a warning says so and the same calls go
through ctypes.
"""
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libsegquant.so")
LIB_DEBUG = os.path.join(HERE, "libsegquant_debug.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsegquant.so")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def calls_path() -> str:
    """Where the compiled calls for this Python and this torch are, or would be."""
    import torch
    tags = (sysconfig.get_config_var("SOABI") or sys.implementation.cache_tag,
            f"torch-{torch.__version__}",
            f"cxx11abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}")
    return os.path.join(HERE, "_sqtorch." + ".".join(tags) + ".so")


def build_calls(force: bool = False):
    """Path of the compiled calls, or None (with a warning) where they cannot be
    built."""
    try:
        return _build_calls(force)
    except (OSError, RuntimeError, subprocess.CalledProcessError) as e:
        if os.path.exists(calls_path()):
            os.remove(calls_path())   # of an older source
        warnings.warn(f"csrc/torch_calls.cpp could not be built ({e}): the operators' calls go "
                      "through ctypes, which costs the host 5 to 15 us more each", RuntimeWarning)
        return None


def _build_calls(force: bool) -> str:
    src = os.path.join(CSRC, "torch_calls.cpp")
    header = os.path.join(INCLUDE, "segquant.h")
    calls = calls_path()
    if (not force and os.path.exists(calls)
            and os.path.getmtime(calls) >= max(os.path.getmtime(src), os.path.getmtime(header))):
        return calls
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = [INCLUDE, os.path.join(home, "include"), os.path.join(cuda, "include"),
            sysconfig.get_paths()["include"]]
    tmp = calls + f".tmp{os.getpid()}"
    try:
        subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
                        "-fvisibility=hidden",
                        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                        *[f"-I{d}" for d in dirs], src, "-o", tmp,
                        "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cuda",
                        "-ltorch_cpu", "-lc10_cuda", "-lc10", "-ldl"], check=True)
        os.replace(tmp, calls)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
    return calls


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib = _build_library(force, verbose, debug)
    build_calls(force)
    return lib


def _build_library(force: bool, verbose: bool, debug: bool) -> str:
    lib = LIB_DEBUG if debug else LIB
    if not force and up_to_date(lib):
        return lib
    objdir = os.path.join(HERE, "_build_debug" if debug else "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *(["-DSQ_DEBUG_BOUNDS"] if debug else []), "-I", INCLUDE,
               "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                debug="--debug" in sys.argv))
