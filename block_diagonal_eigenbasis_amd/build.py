"""Build libdobb.so (HIP, gfx950) in-tree with hipcc, and the host module of the binding with g++.

Every kernel source is compiled for gfx950 only, with packed-fp32 instructions disabled
(-Xclang -target-feature -Xclang -packed-fp32-ops), and linked into one shared library next to this
file; _dobb_host.so (csrc/host_ops.cpp, host code against torch's headers) is linked against it.
build() always recompiles; build(host=False), or this file run with --library, makes libdobb.so alone, which needs
hipcc but neither g++ nor torch's and Python's headers.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libdobb.so")
HOST = os.path.join(PKG, "_dobb_host.so")
BUILD_DIR = os.path.join(PKG, "_build")
SOURCES = ["dobb_api.hip", "dobb_ops.hip", "dobb_layers.hip", "k_norm.hip", "k_fp8.hip", "k_fp8_matmul.hip", "k_moment_fp8.hip", "k_grads.hip", "k_mx4.hip", "k_moment_mx4.hip", "k_basis.hip", "k_cholqr.hip", "k_step.hip", "k_step_g.hip", "k_step_bf16.hip", "k_step_fused.hip", "k_accumulate.hip", "k_refresh.hip", "k_qr.hip", "k_step_rows.hip", "k_step_wide.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17", "-Wall", "-Wno-unused-result",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(PKG, "..", "include")]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj


def _build_host() -> None:
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    inc = [x for d in cpp_extension.include_paths("cuda") for x in ("-isystem", d)]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = HOST + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-fPIC", "-shared", "-std=c++17", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc, "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "host_ops.cpp"), "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch", "-lc10", "-lc10_hip",
           "-L", PKG, "-ldobb", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on host_ops.cpp:\n{r.stderr}")
    os.replace(tmp, HOST)


def build(verbose: bool = False, host: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if host:
        _build_host()
    if verbose:
        print(f"built {LIB} and {HOST}" if host else f"built {LIB}")
    return LIB


if __name__ == "__main__":
    if sys.argv[1:] not in ([], ["--library"]):
        sys.exit("usage: build.py [--library]")
    build(verbose=True, host=not sys.argv[1:])
