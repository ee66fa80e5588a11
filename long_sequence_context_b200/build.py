"""Build libcpattn.so (the C-ABI library) in-tree for sm_100a, and _calls.so,
the C++ side of the Python binding's per-token calls.

    python -m long_sequence_context_b200.build [--force] [--verbose]

Each csrc/*.cu is compiled by nvcc (-gencode arch=compute_100a,code=sm_100a
-O3 -lineinfo) into _build/, then linked into long_sequence_context_b200/
libcpattn.so with the CUDA runtime linked statically.  No vendor math library
is linked: every kernel is this package's own.  csrc/calls.cpp is host code
against PyTorch's headers, compiled by g++ for the torch and Python that are
installed; where that fails the binding does without it.
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libcpattn.so")
CALLS = os.path.join(PKG, "_calls.so")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-O2", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC] + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, (r.stdout + r.stderr)


def _torch():
    """torch's folder and version, without importing it."""
    path = importlib.util.find_spec("torch").submodule_search_locations[0]
    with open(os.path.join(path, "version.py")) as f:
        return path, re.search(r"^__version__ = ['\"](.*)['\"]", f.read(), re.M).group(1)


def calls_tag(torch_version):
    """What a _calls.so is built for: it uses the C++ interfaces of one torch and the C API of one Python."""
    return f"torch {torch_version}, python {sys.version_info[0]}.{sys.version_info[1]}"


def _build_calls(force):
    src, stamp = os.path.join(CSRC, "calls.cpp"), os.path.join(BUILD, "calls.tag")
    torch_dir, version = _torch()
    tag, old = calls_tag(version), None
    if os.path.exists(stamp):
        with open(stamp) as f:
            old = f.read()
    if not (force or old != tag or _stale(CALLS, [src, os.path.join(ROOT, "include", "cpattn.h")])):
        return
    cuda = os.path.dirname(os.path.dirname(NVCC))
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(torch_dir, "include"), "-I", os.path.join(cuda, "include"),
           "-I", sysconfig.get_paths()["include"], f'-DCALLS_TAG="{tag}"', src, "-o", CALLS + ".tmp",
           "-L", os.path.join(torch_dir, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(CALLS + ".tmp", CALLS)
    with open(stamp, "w") as f:
        f.write(tag)


def _try_calls(force):
    try:
        _build_calls(force)
    except (RuntimeError, OSError, AttributeError) as e:  # no compiler, no headers, another torch's headers
        if os.path.exists(CALLS):  # of other sources
            os.remove(CALLS)
        warnings.warn(f"_calls.so was not built, the paged cache's calls go through ctypes: {e}")


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    hdrs = _headers()
    todo = [s for s in srcs
            if force or verbose or _stale(os.path.join(BUILD, os.path.basename(s) + ".o"), [s] + hdrs)]
    logs = []
    if todo:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(todo))) as ex:
            for obj, log in ex.map(lambda s: _compile(s, verbose), todo):
                logs.append(log)
    objs = [os.path.join(BUILD, os.path.basename(s) + ".o") for s in srcs]
    if todo or _stale(LIB, objs):
        cuda_lib = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "lib64")
        cmd = [NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-cudart", "static",
               "-o", LIB] + objs + ["-L" + cuda_lib, "-Xlinker", "-rpath," + cuda_lib]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _try_calls(force)
    if verbose:
        print("\n".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
