"""Builds the libraries in-tree from csrc/: libgemm_bf16.so and libfp8_ops.so with nvcc
for sm_103a, and the Python binding of the latter, _fp8_bind.so, with the host compiler.

The translation units compile in parallel; the CUDA runtime is linked
statically and every symbol except the C ABIs of include/gemm_bf16.h and
include/fp8_ops.h is hidden, so each library loads (and exports its ABI) on a
machine without a GPU.  The libraries need nvcc alone; the binding is built where
torch is installed, after them.
"""
from __future__ import annotations

import hashlib
import os
import platform
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgemm_bf16.so")
FP8_LIB = os.path.join(PKG, "libfp8_ops.so")
FP8_BIND = os.path.join(PKG, "_fp8_bind.so")
BUILD_DIR = os.path.join(PKG, "_build")

SOURCES = ["gemm_bf16_api.cu", "gemm_ws_c1.cu", "gemm_ws_c2.cu", "gemm_nows.cu", "gemm_bf16_noalloc.cu",
           "gemm_repack.cu", "gemm_thin.cu"]
FP8_SOURCES = ["fp8_api.cu", "fp8_gemm.cu", "fp8_quantize.cu", "fp8_norm.cu"]
FP8_BIND_SOURCE = "fp8_bind.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the libraries")


def cxx() -> str:
    for cand in (shutil.which("g++"), shutil.which("c++")):
        if cand:
            return cand
    raise RuntimeError("g++ not found: a host compiler is required to build the Python binding")


def bind_flags() -> tuple:
    """(compile flags, link flags) of the Python binding: torch's headers and libraries."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    comp = ["-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-I", CSRC]
    for path in include:
        comp += ["-isystem", path]
    link = ["-shared", "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda",
            "-lc10", "-lc10_cuda", "-L", PKG, "-lfp8_ops", "-Wl,-rpath,$ORIGIN"]
    return comp, link


def source_digest() -> str:
    """sha256 over every file under csrc/ and include/ (identifies a kernel build)."""
    h = hashlib.sha256()
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            path = os.path.join(d, name)
            if os.path.isfile(path):
                h.update(name.encode())
                with open(path, "rb") as fh:
                    h.update(fh.read())
    return h.hexdigest()


# What decides the GEMM kernel's behaviour on a given problem: its device code
# and the host planner that picks its launch shape (not the public header's
# documentation, the binding or the other kernels).
KERNEL_FILES = ["gemm_ws.cuh", "gemm_common.cuh", "ptx.cuh", "ring_index.h", "gemm_kernels.h", "gemm_ws_c1.cu",
                "gemm_ws_c2.cu", "gemm_bf16_api.cu"]


def kernel_digest() -> str:
    """sha256 over the files in KERNEL_FILES: identifies a measured kernel."""
    h = hashlib.sha256()
    for name in KERNEL_FILES:
        with open(os.path.join(CSRC, name), "rb") as fh:
            h.update(name.encode())
            h.update(fh.read())
    return h.hexdigest()


def _stamp_path() -> str:
    return os.path.join(BUILD_DIR, "stamp.txt")


def _bind_stamp_path() -> str:
    return os.path.join(BUILD_DIR, "bind_stamp.txt")


def torch_version() -> str | None:
    """Version of the installed torch, against which the binding is built; None without one."""
    try:
        import torch
    except ImportError:
        return None
    return torch.__version__


def _nvcc_version(cc: str) -> str:
    try:
        res = subprocess.run([cc, "--version"], capture_output=True, text=True)
        return res.stdout.strip().splitlines()[-1] if res.stdout.strip() else "unknown"
    except OSError:
        return "unknown"


def build_stamp(cc: str | None = None) -> str:
    """What a built library depends on: its sources, the host architecture it
    was linked for, the compiler and the flags.  A library built on another
    machine (an x86_64 build seen on an aarch64 host) never matches."""
    cc = cc or nvcc()
    return "\n".join([source_digest(), "machine=" + platform.machine(), "nvcc=" + _nvcc_version(cc),
                      "flags=" + " ".join(ARCH + FLAGS)])


def bind_stamp() -> str:
    """What the built binding depends on besides."""
    return "\n".join([source_digest(), "machine=" + platform.machine(), f"torch={torch_version()}"])


def _stamped(path: str, stamp: str, *built: str) -> bool:
    if not all(os.path.exists(f) for f in (path, *built)):
        return False
    with open(path) as fh:
        return fh.read().strip() == stamp


def libraries_up_to_date(cc: str | None = None) -> bool:
    return _stamped(_stamp_path(), build_stamp(cc), LIB, FP8_LIB)


def binding_up_to_date() -> bool:
    """Also where there is no torch to build it against."""
    return torch_version() is None or _stamped(_bind_stamp_path(), bind_stamp(), FP8_BIND)


def up_to_date(cc: str | None = None) -> bool:
    return libraries_up_to_date(cc) and binding_up_to_date()


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is not up to date (with `force`, everything) and returns libgemm_bf16.so's path."""
    cc = nvcc()
    libraries = force or not libraries_up_to_date(cc)
    binding = torch_version() is not None and (force or not binding_up_to_date())
    if not libraries and not binding:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and res.stderr:
            sys.stderr.write(res.stderr)
        return obj

    def compile_bind() -> str:
        obj = os.path.join(BUILD_DIR, FP8_BIND_SOURCE.replace(".cpp", ".o"))
        cmd = [cxx(), *bind_flags()[0], "-c", os.path.join(CSRC, FP8_BIND_SOURCE), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on {FP8_BIND_SOURCE}:\n{res.stdout}\n{res.stderr}")
        return obj

    def link(lib: str, cmd: list) -> None:
        tmp = lib + f".tmp{os.getpid()}"
        res = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, lib)

    def stamp(path: str, text: str) -> None:
        with open(path, "w") as fh:
            fh.write(text)

    sources = SOURCES + FP8_SOURCES if libraries else []
    with ThreadPoolExecutor(max_workers=len(sources) + 1) as ex:
        bind_obj = ex.submit(compile_bind) if binding else None
        objs = list(ex.map(compile_one, sources))
        if libraries:
            shared = [cc, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "--exclude-libs,ALL"]
            link(LIB, [*shared, *objs[:len(SOURCES)]])
            link(FP8_LIB, [*shared, *objs[len(SOURCES):]])
            stamp(_stamp_path(), build_stamp(cc))
        if binding:  # its failure leaves the libraries built
            link(FP8_BIND, [cxx(), bind_obj.result(), *bind_flags()[1]])
            stamp(_bind_stamp_path(), bind_stamp())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
