"""Builds the sm_103a attention library in-tree: _build/libattn_fwd.so, and the
CPython module of its norm and cache conveniences: _build/_serve.<versions>.so,
for this interpreter and this torch.  The library needs neither.

nvcc compiles the CUDA sources for sm_103a only and links the CUDA runtime
statically, so the library loads on a machine without a GPU (every CUDA call
then fails cleanly) and needs no libcuda at link time (the TMA descriptor
encoder is looked up through the runtime's driver entry-point query).
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libattn_fwd.so")
SOURCES = [os.path.join(CSRC, "attn_fwd.cu"), os.path.join(CSRC, "attn_bwd.cu"),
           os.path.join(CSRC, "attn_serve.cu")]
# the torch conveniences of the norm and cache calls, as a CPython module
BINDING_SOURCE = os.path.join(CSRC, "serve_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _deps():
    deps = list(SOURCES)
    deps += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return deps


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def binding_path() -> str:
    """The module's file; its name holds what it is compiled against, so that another
    Python or torch gets one of its own."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(OUT_DIR, f"_serve.{sys.implementation.cache_tag}.torch-{torch.__version__}.abi{abi}.so")


def _binding_command(out: str) -> list[str]:
    """g++ on the binding, with the headers and libraries of this interpreter and torch."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
            "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), BINDING_SOURCE, "-o", out,
            "-L", os.path.join(root, "lib"), "-Wl,-rpath," + os.path.join(root, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]


def _binding_fresh(path: str) -> bool:
    deps = [BINDING_SOURCE, __file__] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(p) for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is missing or older than its sources; returns the library's path.
    Without torch the module of torch conveniences is left out."""
    os.makedirs(OUT_DIR, exist_ok=True)
    binding = None
    try:
        path = binding_path()
        if force or not _binding_fresh(path):
            tmp = path + f".tmp{os.getpid()}"
            cmd = _binding_command(tmp)
            binding = (cmd, tmp, path, subprocess.Popen(cmd))  # beside the kernels
    except ImportError as e:
        print(f"no torch ({e}): the library alone is built", file=sys.stderr)
    try:
        return _build_library(force, verbose)
    finally:
        if binding:
            cmd, tmp, path, pr = binding
            if pr.wait() != 0:
                raise subprocess.CalledProcessError(pr.returncode, cmd)
            os.replace(tmp, path)


def _build_library(force: bool, verbose: bool) -> str:
    if not force and os.path.exists(LIB):
        if os.path.getmtime(LIB) >= max(os.path.getmtime(p) for p in _deps()):
            return LIB
    tag = f".tmp{os.getpid()}"
    # one translation unit per source, compiled in parallel, then one link
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(OUT_DIR, os.path.basename(src) + tag + ".o")
        cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
               "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        objs.append(obj)
        procs.append((cmd, subprocess.Popen(cmd)))
    failed = [cmd for cmd, pr in procs if pr.wait() != 0]
    try:
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        tmp = LIB + tag
        subprocess.run([nvcc(), *ARCH, "-shared", *objs, "-o", tmp], check=True)
        os.replace(tmp, LIB)
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
