"""Builds the GDN C-ABI shared library (``libgdn_gb300.so``) with nvcc.

One translation unit per ``csrc/*.cu`` file, compiled in parallel for sm_103a
only, then linked into a shared library next to this file (in-tree, so the
process that loads it is visibly using the CUDA path). The CUDA runtime is
linked statically; the library exports only the ``gdn_*`` C symbols declared in
``include/gdn.h``. ``csrc/marshal.cpp``, the part of the Python binding that is
compiled, becomes an extension module beside the library.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC_DIR = os.path.join(PKG_DIR, "csrc")
INCLUDE_DIR = os.path.join(REPO_DIR, "include")
MARSHAL_SRC = os.path.join(CSRC_DIR, "marshal.cpp")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libgdn_gb300.so")
MARSHAL_PATH = os.path.join(PKG_DIR, "_marshal.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH_FLAGS + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE_DIR, "-I", CSRC_DIR,
]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the GDN library needs the CUDA 13 toolkit")


def _sources():
    return sorted(os.path.join(CSRC_DIR, f) for f in os.listdir(CSRC_DIR) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(INCLUDE_DIR, f) for f in os.listdir(INCLUDE_DIR) if f.endswith(".h")]
    hs += [os.path.join(CSRC_DIR, f) for f in os.listdir(CSRC_DIR) if f.endswith((".cuh", ".h"))]
    return hs


def _stale(lib: str, inputs) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in list(inputs) + [__file__])


def _marshal_stamp() -> str:
    import torch
    return f"{torch.__version__} {sysconfig.get_python_version()}"


def _marshal_stale() -> bool:
    stamp = os.path.join(BUILD_DIR, "marshal.stamp")
    if _stale(MARSHAL_PATH, [MARSHAL_SRC, os.path.join(INCLUDE_DIR, "gdn.h")]) or not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        return f.read() != _marshal_stamp()


def _build_marshal(verbose: bool = False):
    """The extension module, against the installed torch and the library."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    tmp = MARSHAL_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=" + str(int(torch.compiled_with_cxx11_abi())),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", INCLUDE_DIR, MARSHAL_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           LIB_PATH, "-Wl,-rpath," + os.path.join(root, "lib"), "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL_PATH)
    with open(os.path.join(BUILD_DIR, "marshal.stamp"), "w") as f:
        f.write(_marshal_stamp())


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link what has changed, the library and the extension module;
    return the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if force or _stale(LIB_PATH, _sources() + _headers()):
        _build_library(verbose, extra_flags)
    if force or _marshal_stale():
        _build_marshal(verbose)
    return LIB_PATH


def _build_library(verbose: bool, extra_flags):
    nvcc = nvcc_path()
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + ".tmp"
    # The soname lets the extension module find the library beside itself.
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB_PATH), "-o", tmp,
           *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
