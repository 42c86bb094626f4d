"""Builds, in-tree, ``libhstu_attn.so`` (the CUDA library behind include/hstu_attn.h and include/hstu_paged.h,
for sm_100a) and ``_paged_native.so`` (the C++ marshalling of the paged calls for Python)."""
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libhstu_attn.so")
SOURCES = ["hstu_attn.cu", "hstu_paged.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-shared", "--threads", "0", "-I" + INCLUDE, "-I" + CSRC]
MODULE = os.path.join(PKG, "_paged_native.so")
MODULE_SOURCES = ["paged_binding.cpp"]
CXX = os.environ.get("CXX", "g++")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f not in MODULE_SOURCES]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _newer(target, inputs) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def built_for() -> str:
    """What the marshalling module's C++ interface is that of: the torch and the Python it is compiled against."""
    import torch
    return "torch %s, %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def _stamp() -> str:
    return MODULE + ".built_for"


def module_built_for():
    """built_for() of the build that made the module; None if that is not known."""
    try:
        with open(_stamp()) as f:
            return f.read()
    except OSError:
        return None


def build_module(force: bool = False) -> str:
    """Compiles the marshalling module if a source of it is newer, or if it was made for another torch or Python;
    returns its path."""
    sources = [os.path.join(CSRC, s) for s in MODULE_SOURCES]
    if not force and module_built_for() == built_for() and _newer(
            MODULE, sources + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)]):
        return MODULE
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = MODULE + ".tmp%d" % os.getpid()
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I" + INCLUDE, "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-o", tmp] + sources + ["-L" + os.path.join(home, "lib")] + [
           "-l" + lib for lib in ("torch_python", "torch", "torch_cpu", "torch_cuda", "c10", "c10_cuda")]
    subprocess.run(cmd, check=True)
    if os.path.exists(_stamp()):
        os.remove(_stamp())
    os.replace(tmp, MODULE)
    with open(_stamp(), "w") as f:
        f.write(built_for())
    return MODULE


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles what is older than its sources; returns the library's path."""
    build_module(force)
    if not force and up_to_date():
        return LIB
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [NVCC] + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-o", tmp] + [
        os.path.join(CSRC, s) for s in SOURCES]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
