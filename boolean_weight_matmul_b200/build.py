"""Build libmbok.so (sm_100a) in-tree with nvcc.

Every .cu file under csrc/ is compiled to an object in <repo>/_build/ and the
objects are linked into boolean_weight_matmul_b200/libmbok.so (CUDA runtime
linked statically, so the library is self-contained).  Rebuilds only when a
source or header is newer than the library.

build(variant="stamps") builds the profiling library libmbok_stamps.so from
the same sources with MBOK_PHASE_STAMPS defined: the decode lookup kernels
then record per-CTA phase timestamps (read by `bench.py --phase-profile`).

csrc/marshal.cpp, the binding's argument marshalling, becomes the extension
module boolean_weight_matmul_b200/_marshal.<Python ABI>.torch-<version>.so (C++,
against torch's headers, so that each pair of versions has its own).
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libmbok.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
VARIANTS = {"": ("libmbok.so", []), "stamps": ("libmbok_stamps.so", ["-DMBOK_PHASE_STAMPS"])}

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-I" + INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the MBOK library needs the CUDA toolkit to build")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, verbose: bool, out_dir: str = BUILD_DIR, extra=()) -> str:
    obj = os.path.join(out_dir, os.path.basename(src) + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + list(extra) + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def marshal_path() -> str:
    """The extension module of this Python and this torch, whose ABIs it is
    compiled for."""
    import torch
    return os.path.join(HERE, f"_marshal.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def build_marshal(force: bool = False) -> str:
    """Compile the extension module; returns its path."""
    path = marshal_path()
    deps = [MARSHAL_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps):
        return path
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = path + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"]]
    for d in (os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include")):
        cmd += ["-isystem", d]
    cmd += [MARSHAL_SRC, "-o", tmp, "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
            "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, variant: str = "") -> str:
    """Compile and link libmbok.so (or a profiling variant) and the marshalling
    module; returns the library's path."""
    build_marshal(force)
    name, extra = VARIANTS[variant]
    lib = os.path.join(HERE, name)
    out_dir = os.path.join(BUILD_DIR, variant) if variant else BUILD_DIR
    if not force and up_to_date(lib):
        return lib
    os.makedirs(out_dir, exist_ok=True)
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, out_dir, extra), srcs))
    tmp = lib + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
