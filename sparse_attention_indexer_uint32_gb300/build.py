"""Builds ``libtopkidx.so`` (the CUDA library) in-tree with nvcc for sm_103a, and
the module ``_tensor_calls``, which makes some of its calls straight from tensors.

Usage: ``python -m sparse_attention_indexer_uint32_gb300.build [--verbose]``.
The translation units are compiled in parallel, those of the library linked
into one shared library next to this file.  Nothing is installed into
site-packages.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBRARY = os.path.join(PKG, "libtopkidx.so")
SOURCES = ["topk_kernels.cu", "topk_stream.cu", "topk_warp.cu", "topk_split.cu", "topkidx_api.cu", "topk_noalloc.cu",
           "serve_tables.cu", "serve_append.cu", "index_append.cu", "index_scores.cu",
           "attend_latent.cu", "attend_prompt.cu", "attend_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtopkidx.so")
    return path


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "topkidx.h"), __file__]
    return max(os.path.getmtime(f) for f in files)


def tensor_calls_path() -> str:
    """The module ``_tensor_calls`` for the running torch and Python.

    It reads their objects where this version has them, so the file is named by
    both: one that was built for another version is not found, and not loaded.
    """
    import torch

    return os.path.join(PKG, f"_tensor_calls.torch-{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def _old(path: str, force: bool) -> bool:
    return force or not os.path.exists(path) or os.path.getmtime(path) < _deps_mtime()


def _build_tensor_calls(force: bool) -> None:
    """The CPython module, against the headers and libraries of the torch that imports it."""
    path = tensor_calls_path()
    if not _old(path, force):
        return
    import torch

    root = os.path.dirname(torch.__file__)
    include = os.path.join(root, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = path + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-I", include,
           "-I", os.path.join(include, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(cuda, "include"), os.path.join(CSRC, "tensor_calls.cpp"), "-o", tmp,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for tensor_calls.cpp:\n{res.stderr}")
    os.replace(tmp, path)


def _build_library(verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *common, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stderr}")
        if verbose and res.stderr:
            sys.stderr.write(res.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIBRARY + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIBRARY)


def build(verbose: bool = False, force: bool = False) -> str:
    """The library's path; what fails in the module is raised once the library, which works without it, is there."""
    with concurrent.futures.ThreadPoolExecutor(1) as ex:
        calls = ex.submit(_build_tensor_calls, force)
        if _old(LIBRARY, force):
            _build_library(verbose)
        calls.result()
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
