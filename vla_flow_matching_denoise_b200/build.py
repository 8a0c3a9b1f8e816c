"""Builds the C-ABI shared library in-tree with nvcc for sm_100a.

    python -m vla_flow_matching_denoise_b200.build [--force]

Output: vla_flow_matching_denoise_b200/libfm_expert.so (C ABI declared in
include/fm_expert.h and include/fm_ops.h) and _ops.so beside it (the Python
module that calls include/fm_ops.h on torch tensors; host code only, linked to
the library).  Rebuilds only what is older than its sources, and _ops.so where
another Python or torch built it.  Without a CUDA build of torch there is no
_ops.so; the library and its numpy binding need neither.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfm_expert.so")
OPS = os.path.join(PKG, "_ops.so")
SOURCES = ["fm_api.cu", "fm_prep.cu", "fm_time.cu", "fm_step.cu", "fm_batch.cu", "fm_attn.cu", "fm_noalloc.cu",
           "fm_ops.cu", "fm_ops_gemm.cu"]
HEADERS = ["fm_internal.h", "fm_batch.h", "fm_launch.h", "fm_ptx.cuh", "fm_ops_check.h", "fm_ops_math.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put /usr/local/cuda/bin on PATH)")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps += [os.path.join(ROOT, "include", f) for f in ("fm_expert.h", "fm_ops.h")]
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(p) > t for p in deps)


def _ops_stale(key: str) -> bool:
    """Whether _ops.so is missing, older than its sources or built for something
    else than `key` (a text that it holds)."""
    deps = [os.path.join(CSRC, "fm_ops_torch.cpp"), os.path.join(ROOT, "include", "fm_ops.h"),
            os.path.join(ROOT, "include", "fm_expert.h"), os.path.abspath(__file__)]
    if not os.path.exists(OPS) or any(os.path.getmtime(p) > os.path.getmtime(OPS) for p in deps):
        return True
    with open(OPS, "rb") as f:
        return key.encode() + b"\0" not in f.read()


def _build_ops(force: bool) -> None:
    """The torch module of the operators (g++, a few headers of torch; needs LIB)."""
    try:
        import torch
    except ImportError:
        torch = None
    if torch is None or torch.version.cuda is None:
        print("no CUDA build of torch: _ops.so (the operators on torch tensors) is not built", file=sys.stderr)
        return
    key = f"fm_ops for {sys.implementation.cache_tag}, torch {torch.__version__}"
    if not force and not _ops_stale(key):
        return
    src = os.path.join(CSRC, "fm_ops_torch.cpp")
    t = os.path.dirname(os.path.abspath(torch.__file__))
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DFM_OPS_BUILT_FOR="{key}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(t, "include"), "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include"),
           "-o", OPS + ".tmp", src, "-L", PKG, "-l:libfm_expert.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(t, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(OPS + ".tmp", OPS)


def build(force: bool = False, verbose: bool = False) -> str:
    _build_lib(force, verbose)
    _build_ops(force)
    return LIB


def _build_lib(force: bool, verbose: bool) -> str:
    if not force and not _stale():
        return LIB
    cmd = [nvcc_path(), "-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-shared", "-diag-suppress", "177",
           "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp"]
    cmd += [os.path.join(CSRC, f) for f in SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
