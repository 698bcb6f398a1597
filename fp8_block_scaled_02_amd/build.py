"""Compile libfp8blk.so and libfp8attn.so (HIP, gfx950) in-tree with hipcc.

The libraries are the product's compute path: every hot-path step runs in
the kernels under csrc/ (the linear layers, libfp8blk.so) and csrc/attention/
(the attention side of a decode step, libfp8attn.so).  Compiled with
packed-FP32 instructions disabled.
"""
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp8blk.so")
ATTN_LIB = os.path.join(HERE, "libfp8attn.so")
ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc"), "hipcc"):
        if os.path.sep not in c or os.path.exists(c):
            return c
    return "hipcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def attn_sources():
    return sorted(glob.glob(os.path.join(CSRC, "attention", "*.hip")))


def build(verbose: bool = False) -> str:
    _compile(ATTN_LIB, attn_sources(), verbose)
    return _compile(LIB, sources(), verbose)


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
    print(build(verbose=True))
    sys.exit(0)
