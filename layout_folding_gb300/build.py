"""Build liblayoutfold.so in-tree with nvcc for sm_103a (no torch extension
machinery: the library is a plain C-ABI shared object), and the compiled part of
its Python binding with g++.  The binding is optional: what keeps it from being built
is said and the library is built without it."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

from .compiled import PATH as BINDING_PATH

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "liblayoutfold.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]
# LAYOUTFOLD_NVTX=1 at build time: an NVTX range around every C-ABI call (header-only NVTX 3)
if os.environ.get("LAYOUTFOLD_NVTX", "0") not in ("", "0"):
    CFLAGS.append("-DLF_NVTX")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _binding_command(out):
    """g++ for the compiled part of the Python binding, or None without the headers of
    PyTorch or Python (the ctypes part does every call then)."""
    try:
        import torch
    except ImportError:
        return None
    base = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)))
    python = sysconfig.get_paths()["include"]
    nvcc = shutil.which(NVCC)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include") if nvcc else ""
    if not (os.path.exists(os.path.join(base, "include", "torch", "csrc", "autograd", "python_variable.h"))
            and os.path.exists(os.path.join(python, "Python.h"))
            and os.path.exists(os.path.join(cuda, "cuda_runtime_api.h"))):
        return None
    return [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE, "-I",
            os.path.join(base, "include"), "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"), "-I",
            python, "-I", cuda, BINDING_SRC, "-o", out, "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _older(path, deps):
    """Whether `path` is missing or older than one of deps."""
    return not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps)


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _library_up_to_date() -> bool:
    return not _older(LIB_PATH, _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                      + _headers())


def _binding_up_to_date() -> bool:
    """None is up to date where none can be built; one that is there is not, for that."""
    if not _older(BINDING_PATH, [BINDING_SRC] + _headers()):
        return True
    return not glob.glob(os.path.join(LIB_DIR, "_binding*.so")) and _binding_command(BINDING_PATH) is None


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def _start_binding(out, verbose):
    """g++ at work on the compiled part of the binding, or None where there is none: the
    Python functions do every call then, and the library is built all the same."""
    cmd = _binding_command(out)
    if cmd is None:
        print("no headers of PyTorch or Python: the compiled part of the binding is not built", file=sys.stderr)
        return None
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:
        print("%s: the compiled part of the binding is not built" % e, file=sys.stderr)
        return None


def _finish_binding(p, out, verbose):
    """Puts the binding in its place, and takes away those that are out of date (for
    another PyTorch or Python among them: the library may have changed under them)."""
    text = p.communicate()[0] if p else b""
    if p and (verbose or p.returncode != 0):
        sys.stderr.write(text.decode(errors="replace"))
    for path in glob.glob(os.path.join(LIB_DIR, "_binding*.so")):
        os.remove(path)
    if p and p.returncode == 0:
        os.replace(out, BINDING_PATH)
    elif p:
        print("%s failed: the compiled part of the binding is not built" % p.args[0], file=sys.stderr)
        if os.path.exists(out):
            os.remove(out)


def _build_library(verbose, ptxas_info):
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        objs.append(obj)
        cmd = [NVCC, *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or ptxas_info or p.returncode != 0):
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every .cu in csrc/ (in parallel) and link liblayoutfold.so; beside it the
    compiled part of the Python binding, where this machine can build it."""
    library, binding = force or not _library_up_to_date(), force or not _binding_up_to_date()
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    p = _start_binding(tmp, verbose) if binding else None
    try:
        if library:
            _build_library(verbose, ptxas_info)
    finally:
        if binding:
            _finish_binding(p, tmp, verbose)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
