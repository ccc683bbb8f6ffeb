"""Build libmxq.so (the sm_100a CUDA library) in-tree with nvcc, and
_torch_ops.so, the torch calls and autograd nodes in C++ that use it, with g++.

The library is one translation unit (csrc/mxq.cu includes every kernel) so
that the device status word is a single symbol without relocatable device
code. The CUDA runtime is linked statically; the stream handles passed in by
PyTorch are driver objects and work across runtimes.
"""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmxq.so")
TORCH_SRC = os.path.join(HERE, "csrc_torch", "moe_ops.cpp")
TORCH_OPS = os.path.join(HERE, "_torch_ops.so")
TORCH_OPS_KEY = TORCH_OPS + ".key"  # the torch and Python that it was built against

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-shared", "-Xcompiler", "-fPIC,-O2",
         "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=true",
         "-cudart", "static", "--expt-relaxed-constexpr"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)) + [os.path.join(INCLUDE, "mxq.h")]


def _up_to_date(out, srcs):
    return os.path.exists(out) and all(os.path.getmtime(out) >= os.path.getmtime(s) for s in srcs)


def _torch_key():
    """What a module compiled against torch's C++ classes is bound to."""
    import torch
    return "\n".join((torch.__version__, torch.version.git_version, str(torch._C._GLIBCXX_USE_CXX11_ABI),
                      sysconfig.get_config_var("SOABI")))


def _built_key():
    try:
        with open(TORCH_OPS_KEY) as f:
            return f.read()
    except OSError:
        return None


def build_torch_ops(force=False, verbose=False):
    """_torch_ops.so: host code only, against torch's headers and libmxq.so."""
    if (not force and _built_key() == _torch_key()
            and _up_to_date(TORCH_OPS, [TORCH_SRC, os.path.join(INCLUDE, "mxq.h")])):
        return TORCH_OPS
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-DTORCH_EXTENSION_NAME=_torch_ops",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in inc[:1]), *(f"-isystem{d}" for d in inc[1:]), TORCH_SRC, "-o", TORCH_OPS + ".tmp",
           f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch",
           "-ltorch_python", f"-L{HERE}", "-l:libmxq.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(TORCH_OPS + ".tmp", TORCH_OPS)
    with open(TORCH_OPS_KEY, "w") as f:
        f.write(_torch_key())
    return TORCH_OPS


def build(force=False, verbose=False, extra=()):
    lib = build_library(force, verbose, extra)
    build_torch_ops(force, verbose)
    return lib


def build_library(force=False, verbose=False, extra=()):
    if not force and _up_to_date(LIB, sources()):
        return LIB
    cmd = [NVCC, *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, *extra,
           os.path.join(CSRC, "mxq.cu"), "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "-v" in sys.argv else []
    print(build(force=True, verbose=True, extra=extra))
