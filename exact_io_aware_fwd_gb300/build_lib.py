"""Builds libfa_sm103.so (the C-ABI library) in-tree with nvcc for sm_103a, and the compiled
Python binding of the operators around attention (_serving_binding.*.so) with g++.

The translation units are compiled in parallel into ``<repo>/_build`` and linked into
``exact_io_aware_fwd_gb300/libfa_sm103.so``.  A rebuild happens only when a source or header is
newer than the library (or when ``force=True``).  The binding compiles next to them; it belongs to
the PyTorch and the Python it was built with, whose versions are in its name.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

import torch

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libfa_sm103.so")


def binding_path(torch_version: str, suffix: str) -> str:
    """The binding's file for a PyTorch version and Python's suffix of extension modules."""
    return os.path.join(PKG_DIR, f"_serving_binding.torch-{torch_version}{suffix}")


BINDING_PATH = binding_path(torch.__version__, sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_SOURCE = os.path.join(CSRC, "serving_binding.cpp")
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_bwd_dq.cu", "fa_block_sparse.cu", "fa_noalloc.cu",
           "fa_serving.cu", "fa_rope.cu", "fa_paged.cu", "fa_paged_mma.cu"]
HEADERS = [os.path.join(CSRC, "sm103.cuh"), os.path.join(CSRC, "fa_internal.h"),
           os.path.join(CSRC, "fa_host.h"), os.path.join(CSRC, "fa_paged.h"),
           os.path.join(CSRC, "paged_plan.cuh"), os.path.join(CSRC, "paged_rows.cuh"),
           os.path.join(ROOT, "include", "fa.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
          "-I", os.path.join(ROOT, "include")]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or install the CUDA toolkit)")


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_command(out):
    home = os.path.dirname(os.path.abspath(torch.__file__))
    include = os.path.join(home, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    dirs = [include, os.path.join(include, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
            os.path.join(ROOT, "include")]
    libs = os.path.join(home, "lib")
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[x for d in dirs for x in ("-isystem", d)], BINDING_SOURCE, "-o", out, "-L", libs,
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
            "-Wl,-rpath," + libs]


def build_binding(force: bool = False) -> str:
    """Compile the Python binding of the operators around attention; returns its path."""
    if not force and not _stale(BINDING_PATH, [BINDING_SOURCE, HEADERS[-1], __file__]):
        return BINDING_PATH
    tmp = BINDING_PATH + f".{os.getpid()}.tmp"
    cmd = _binding_command(tmp)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("compiling serving_binding.cpp failed")
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          defines: dict | None = None, out_path: str | None = None) -> str:
    """Compile and link the library; returns its path.

    ``defines`` (name -> value) are passed as -D flags (the kernels' tuning parameters) and
    ``out_path`` places the library elsewhere than the package directory.
    """
    nvcc = _nvcc()
    lib_path = out_path or LIB_PATH
    tag = "" if not defines else "_" + "_".join(f"{k}{v}" for k, v in sorted(defines.items()))
    build_dir = os.path.join(BUILD_DIR, tag.strip("_") or "default")
    os.makedirs(build_dir, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    if not force and not _stale(lib_path, srcs + HEADERS + [__file__]):
        if out_path is None:
            build_binding()
        return lib_path
    objs = [os.path.join(build_dir, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    extra += [f"-D{k}={v}" for k, v in (defines or {}).items()]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc, *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        binding = ex.submit(build_binding, force) if out_path is None else None
        results = list(ex.map(compile_one, zip(srcs, objs)))
        if binding is not None:
            binding.result()
    for cmd, r in results:
        if verbose or ptxas_info or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {cmd[-3]}")
    tmp = lib_path + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("linking libfa_sm103.so failed")
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
