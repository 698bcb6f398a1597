"""Compile libfp8blk.so, libfp8attn.so and libfp8moe.so (HIP, gfx950) in-tree
with hipcc.

The libraries are the product's compute path: every hot-path step runs in
the kernels under csrc/ (the linear layers, libfp8blk.so), csrc_attention/
(the attention side of a decode step, libfp8attn.so, and the host code of its
Python calls, _attn_binding.so, against torch's headers) and csrc_moe/ (expert
routing and the layers in 8-bit integers, libfp8moe.so and _moe_binding.so).
Compiled with packed-FP32 instructions disabled.
"""
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ATTN_CSRC = os.path.join(HERE, "csrc_attention")
LIB = os.path.join(HERE, "libfp8blk.so")
ATTN_LIB = os.path.join(HERE, "libfp8attn.so")
ATTN_BINDING = os.path.join(HERE, "_attn_binding.so")
MOE_CSRC = os.path.join(HERE, "csrc_moe")
MOE_LIB = os.path.join(HERE, "libfp8moe.so")
MOE_BINDING = os.path.join(HERE, "_moe_binding.so")
ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc"), "hipcc"):
        if os.path.sep not in c or os.path.exists(c):
            return c
    return "hipcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def attn_sources():
    return sorted(glob.glob(os.path.join(ATTN_CSRC, "*.hip")))


def moe_sources():
    return sorted(glob.glob(os.path.join(MOE_CSRC, "*.hip")))


def build(verbose: bool = False) -> str:
    """The linear layers and the attention side.  libfp8blk.so first: it needs
    hipcc alone, and is there also where the binding's compiler or torch's
    headers are not."""
    _compile(LIB, sources(), verbose)
    _compile(ATTN_LIB, attn_sources(), verbose)
    _compile_binding(ATTN_BINDING, ATTN_CSRC, "fp8attn", verbose)
    return LIB


def build_moe(verbose: bool = False) -> str:
    """Expert routing and the layers in 8-bit integers."""
    _compile(MOE_LIB, moe_sources(), verbose)
    _compile_binding(MOE_BINDING, MOE_CSRC, "fp8moe", verbose)
    return MOE_LIB


def build_all(verbose: bool = False) -> str:
    build(verbose)
    build_moe(verbose)
    return LIB


def _compile_binding(binding: str, csrc: str, lib: str, verbose: bool) -> None:
    """Host code only, with the system's C++ compiler.  torch's libraries are
    in the process when the module is imported; the library of the calls lies
    beside it."""
    import torch
    root = os.path.dirname(torch.__file__)
    tmp = binding + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           os.path.join(csrc, "binding.cpp"), "-o", tmp,
           "-L" + HERE, "-l" + lib, "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, binding)


def _compile(lib: str, srcs, verbose: bool) -> str:
    tmp = lib + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-Wall", "-Wno-unused-command-line-argument",
           "-I", os.path.join(os.path.dirname(HERE), "include"),
           "-o", tmp] + srcs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build_all(verbose=True))
    sys.exit(0)
