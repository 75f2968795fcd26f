"""Build libmetis.so in-tree with hipcc for gfx950, and _tensors.so.

Usage: python -m spectral_split_quantized_amd.build
"""

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
OUT = os.path.join(HERE, "libmetis.so")
TENSORS_OUT = os.path.join(HERE, "_tensors.so")

# translation units and their extra flags: the register-dequant GEMM is
# scheduled for instruction-level parallelism (its expansion instructions
# must interleave with the matrix instructions of the same wave); the rest
# keeps the default strategy
UNITS = [
    ("metis.hip", []),
    ("gemm_big.hip", ["-mllvm", "-amdgpu-sched-strategy=iterative-ilp"]),
]

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # keep every binary32 rounding of the quantiser explicit
    "-ffp-contract=off",
    # packed FP32 instructions are avoided on this target
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def build_tensors(verbose=False):
    """_tensors.so: the extension that reads tensor lists (host code against
    torch's headers)."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    cmd = [hipcc, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, os.path.join(CSRC, "tensors.cpp"),
           "-I", sysconfig.get_paths()["include"]]
    cmd += [a for d in include_paths() for a in ("-isystem", d)]
    cmd += [a for d in library_paths() for a in ("-L", d)] + ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    tmp = TENSORS_OUT + ".tmp"
    _run(cmd + ["-o", tmp], verbose)
    os.replace(tmp, TENSORS_OUT)
    return TENSORS_OUT


def build(verbose=False):
    """libmetis.so, then _tensors.so: the library needs no torch, so a failure
    against torch's headers leaves it built."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    os.makedirs(OBJ, exist_ok=True)
    objs = []
    for src, extra in UNITS:
        obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
        _run([hipcc] + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj], verbose)
        objs.append(obj)
    tmp = OUT + ".tmp"
    _run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + ["-o", tmp], verbose)
    os.replace(tmp, OUT)
    build_tensors(verbose)
    return OUT


# Host code under AddressSanitizer and UndefinedBehaviorSanitizer (the device
# code is built as usual): each sanitizer option applies to the host pass only.
HOST_SANITIZE = [
    "-Xarch_host", "-fsanitize=address",
    "-Xarch_host", "-fsanitize=undefined",
    "-Xarch_host", "-fno-sanitize-recover=all",
    "-Xarch_host", "-fno-omit-frame-pointer",
]
SAN_OUT = os.path.join(OBJ, "libmetis_san.so")


def build_host_sanitized(verbose=False):
    """_build/libmetis_san.so: the C-ABI translation unit (metis.hip, all of
    the host-side argument checking, workspace carving and scheduling) with
    host ASan + UBSan, linked with the regular GEMM unit.  Load it with
    METIS_LIBRARY set to its path and the ASan runtime preloaded; only calls
    that need no GPU can run where there is none."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    os.makedirs(OBJ, exist_ok=True)
    gemm_obj = os.path.join(OBJ, "gemm_big.o")
    if not os.path.exists(gemm_obj):
        build(verbose)
    obj = os.path.join(OBJ, "metis_san.o")
    flags = [f for f in FLAGS if f != "-O3"] + ["-O1", "-g"] + HOST_SANITIZE
    _run([hipcc] + flags + ["-c", os.path.join(CSRC, "metis.hip"), "-o", obj], verbose)
    tmp = SAN_OUT + ".tmp"
    _run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC"] + HOST_SANITIZE[:4] + [obj, gemm_obj, "-o", tmp],
         verbose)
    os.replace(tmp, SAN_OUT)
    return SAN_OUT


if __name__ == "__main__":
    build(verbose=True)
    print("built", OUT)
    sys.exit(0)
