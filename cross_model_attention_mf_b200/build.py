"""Build libmf.so (the C-ABI library) in-tree for sm_100a with nvcc, and _mf_bind.so (the Python
side of the paged cache's calls) with g++ against the installed PyTorch's headers.

This file imports nothing from the package (whose import needs the built library): load it
by path with `load_builder()` of the repository's `__graft_entry__`, or run it as a script."""
import glob
import importlib.util
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmf.so")
BIND = os.path.join(HERE, "_mf_bind.so")
BIND_SOURCE = os.path.join(HERE, "csrc", "bind.cpp")
HEADER = os.path.join(ROOT, "include", "mf.h")
NVCC_FLAGS = ["-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
              "-shared", "--threads", "0", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in deps)


def _run(cmd, target, verbose):
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(target + ".tmp", target)


def _bind_command():
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    lib = os.path.join(torch, "lib")
    return ["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-fvisibility=hidden",
            "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), "-o", BIND + ".tmp", BIND_SOURCE,
            "-L", lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force=False, verbose=False):
    if force or _stale(LIB, sources() + glob.glob(os.path.join(HERE, "csrc", "*.cuh")) + [HEADER]):
        _run(["nvcc", *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp", *sources()], LIB, verbose)
    if force or _stale(BIND, [BIND_SOURCE, HEADER]):
        _run(_bind_command(), BIND, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
