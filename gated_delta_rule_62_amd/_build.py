"""Builds the HIP library ``libkda.so`` in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_PATH = os.path.join(PKG_DIR, "libkda.so")
CALLS_PATH = os.path.join(PKG_DIR, "_serving_calls.so")
SOURCES = ["kda_kernel.hip", "kda_api.cpp", "step_kernel.hip", "la_kernel.hip",
           "attn_kernel.hip", "ops_api.cpp"]

# Packed fp32 VALU forms are disabled for every device compile; hipcc's host pass
# warns that it does not know the feature, which is harmless.
HIP_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Wall", "-Wno-unused-function"]


def rocm() -> str:
    return os.environ.get("ROCM_PATH", "/opt/rocm")


def hipcc() -> str:
    return os.path.join(rocm(), "bin", "hipcc")


def build_serving_calls(verbose: bool = False) -> str | None:
    """Compile the serving bindings' calls (host code over torch's headers, with ROCm's own
    compiler); None without torch, whose tensors they take."""
    import sysconfig

    try:
        import torch
    except ImportError:
        print("torch is not installed: the serving operators' calls from Python are not built",
              flush=True)
        return None
    root = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    tmp = CALLS_PATH + ".tmp%d" % os.getpid()
    cmd = [os.path.join(rocm(), "bin", "amdclang++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(rocm(), "include"),
           "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, "serving_calls.cpp"),
           "-o", tmp, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALLS_PATH)
    return CALLS_PATH


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link ``libkda.so``, which needs ROCm alone, then the serving
    bindings' calls (always recompiles)."""
    objs = []
    for src in SOURCES:
        obj = os.path.join(CSRC, os.path.splitext(src)[0] + ".o")
        lang = ["-x", "hip"]
        cmd = [hipcc()] + HIP_FLAGS + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    build_serving_calls(verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
