"""Builds libbbpe.so (the C-ABI library) in this directory with hipcc for
gfx950, and, where torch is installed, _serving.so, the binding's short way to
it from torch.  Usage: python -m byte_level_bpe_amd.build"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libbbpe.so")
SERVING = os.path.join(HERE, "_serving.so")
BUILD = os.path.join(HERE, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = os.environ.get("BBPE_ARCH", "gfx950")

SOURCES = ["bbpe_tables.cpp", "bbpe_front.hip", "bbpe_split.hip", "bbpe_back.hip",
           "bbpe_encode.hip", "bbpe_decode.hip", "bbpe_paging.hip", "bbpe_rope.hip",
           "bbpe_attention.hip", "bbpe_scores.hip", "bbpe_distill.hip"]
COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
          "-I" + os.path.join(HERE, "..", "include")]
HIPFLAGS = ["--offload-arch=" + ARCH, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-munsafe-fp-atomics"]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    path = os.path.join(CSRC, src)
    if src.endswith(".hip"):
        cmd = [HIPCC, "-x", "hip"] + HIPFLAGS + COMMON + ["-c", path, "-o", obj]
    else:
        cmd = ["g++"] + COMMON + ["-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed: %s\n%s\n%s" % (" ".join(cmd), r.stdout, r.stderr))
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _serving() -> None:
    """bbpe_torch.cpp against the installed torch's headers and libraries."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = SERVING + ".tmp"
    cmd = (["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, os.path.join(CSRC, "bbpe_torch.cpp"),
            "-I" + sysconfig.get_paths()["include"]] + ["-isystem" + p for p in include_paths(device_type="cuda")] +
           ["-L" + p for p in library_paths(device_type="cuda")] +
           ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip", "-o", tmp])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed: %s\n%s" % (" ".join(cmd), r.stderr))
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    os.replace(tmp, SERVING)


def build(verbose: bool = False) -> str:
    """The library first: it needs no torch, and no failure of the extension takes it away."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES) + 1)) as ex:
        serving = ex.submit(_serving) if importlib.util.find_spec("torch") else None
        objs = list(ex.map(_compile, SOURCES))
        tmp = OUT + ".tmp"
        # -z defs: a kernel declared but not defined fails the link here, not at load
        cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-Wl,-z,defs", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed: %s\n%s" % (" ".join(cmd), r.stderr))
        os.replace(tmp, OUT)
        if verbose:
            print("built", OUT)
        if serving is None:
            sys.stderr.write("torch is not installed: _serving.so, for the operators on torch tensors, is not built\n")
        else:
            serving.result()
    return OUT


if __name__ == "__main__":
    build(verbose=True)
