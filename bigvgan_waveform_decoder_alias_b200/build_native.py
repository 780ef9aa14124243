"""Build libbv.so (the CUDA library) in-tree with nvcc for sm_100a, and the
tensor marshalling of its token operators (_tokens, C++ against torch; not built
where there is no torch: the library alone serves C callers)."""
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbv.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr", "--threads", "0",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


BINDING_SRC = os.path.join(CSRC, "token_binding.cpp")
BINDING = os.path.join(PKG, "_tokens" + sysconfig.get_config_var("EXT_SUFFIX"))


def _older(out, deps):
    return not os.path.exists(out) or any(os.path.getmtime(d) > os.path.getmtime(out) for d in deps)


def _stale():
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _built_for(mark: str) -> bool:
    """Does the binding carry this mark of the torch it was built against?"""
    with open(BINDING, "rb") as f:
        return mark.encode() in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    import torch
    mark = f"built for torch {torch.__version__}."
    if not force and not _older(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "bv.h")]) and \
            _built_for(mark):
        return BINDING
    base = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    inc = [os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_path("include"), INCLUDE]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-DTORCH_EXTENSION_NAME=_tokens", f'-DBUILT_FOR="{mark}"', *(f"-isystem{d}" for d in inc), BINDING_SRC,
           "-o", BINDING + ".tmp", "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if force or _stale():
        _build_library(verbose, extra)
    try:
        import torch  # noqa: F401
    except ImportError:
        print("no torch: the binding of the token operators is not built", file=sys.stderr)
    else:
        build_binding(force, verbose)
    return LIB


def _build_library(verbose: bool, extra) -> None:
    nvcc = os.environ.get("NVCC", "nvcc")
    cmd = [nvcc, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-o", LIB + ".tmp", *sources()]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(LIB + ".tmp", LIB)


if __name__ == "__main__":
    extra = [a for a in sys.argv[1:] if a.startswith("-X") or a.startswith("--")]
    extra = [a for a in extra if a != "--force"]
    print(build(force="--force" in sys.argv, verbose=True, extra=extra))
