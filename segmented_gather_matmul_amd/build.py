"""Build the C-ABI library ``liblora_sgmv.so`` in-tree with hipcc for gfx950, and with g++ the
small module of the decode-step binding's argument checks (``_step_args``).

    python -m segmented_gather_matmul_amd.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblora_sgmv.so")
SOURCES = [os.path.join(CSRC, "lora_kernels.hip"), os.path.join(CSRC, "lora_pool.hip"),
           os.path.join(CSRC, "lora_step.hip"), os.path.join(CSRC, "lora_host.cpp")]
HEADERS = [os.path.join(INCLUDE, "lora_sgmv.h"), os.path.join(INCLUDE, "lora_step.h"),
           os.path.join(CSRC, "lora_internal.hpp")]
ARCH = "gfx950"
ARGS_LIB = os.path.join(PKG, "_step_args.so")
ARGS_SOURCE = os.path.join(CSRC, "step_args.cpp")


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def flags() -> list[str]:
    return ["-O3", "-std=c++17", "-fPIC", "-shared", f"--offload-arch={ARCH}",
            # Packed FP32 instructions stay off: plain float code is compiled to scalar FP32 ops.
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            # Leading scalar kernel arguments (up to four; only the hand-off kernel has any
            # before its argument block) arrive preloaded in scalar registers.
            "-mllvm", "-amdgpu-kernarg-preload-count=4",
            "-Wall", "-Wno-unused-function", f"-I{INCLUDE}", f"-I{CSRC}"]


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    cmd = [hipcc(), *flags(), *SOURCES, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed building liblora_sgmv.so")
    os.replace(tmp, LIB)
    build_args(verbose)
    return LIB


def build_args(verbose: bool = False) -> str:
    import sysconfig

    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    tmp = ARGS_LIB + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f"-I{sysconfig.get_paths()['include']}",
           "-isystem", inc, f"-I{INCLUDE}", ARGS_SOURCE, "-o", tmp, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10",
           f"-Wl,-rpath,{lib}"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building _step_args.so")
    os.replace(tmp, ARGS_LIB)
    return ARGS_LIB


def stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(ARGS_LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in SOURCES + HEADERS) or \
        any(os.path.getmtime(p) > os.path.getmtime(ARGS_LIB) for p in [ARGS_SOURCE, HEADERS[0], HEADERS[1]])


if __name__ == "__main__":
    print(build(verbose=True))
