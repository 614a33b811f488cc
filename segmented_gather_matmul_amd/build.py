"""Build the C-ABI library ``liblora_sgmv.so`` in-tree with hipcc for gfx950, and with g++ the
small module of the decode-step binding's argument checks (``_step_args``).

    python -m segmented_gather_matmul_amd.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblora_sgmv.so")
SOURCES = [os.path.join(CSRC, "lora_kernels.hip"), os.path.join(CSRC, "lora_pool.hip"),
           os.path.join(CSRC, "lora_step.hip"), os.path.join(CSRC, "lora_quant.hip"), os.path.join(CSRC, "lora_sample.hip"),
           os.path.join(CSRC, "lora_host.cpp")]
PUBLIC_HEADERS = [os.path.join(INCLUDE, "lora_sgmv.h"), os.path.join(INCLUDE, "lora_step.h"),
                  os.path.join(INCLUDE, "lora_quant.h"), os.path.join(INCLUDE, "lora_sample.h")]
HEADERS = PUBLIC_HEADERS + [os.path.join(CSRC, "lora_internal.hpp"), os.path.join(CSRC, "step_device.hpp")]
ARCH = "gfx950"
ARGS_LIB = os.path.join(PKG, "_step_args.so")
ARGS_SOURCE = os.path.join(CSRC, "step_args.cpp")


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def flags() -> list[str]:
    return ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
            # Packed FP32 instructions stay off: plain float code is compiled to scalar FP32 ops.
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            # Leading scalar kernel arguments (up to four; only the hand-off kernel has any
            # before its argument block) arrive preloaded in scalar registers.
            "-mllvm", "-amdgpu-kernarg-preload-count=4",
            "-Wall", "-Wno-unused-function", f"-I{INCLUDE}", f"-I{CSRC}"]


def _hipcc(args, verbose):
    cmd = [hipcc(), *flags(), *args]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed building liblora_sgmv.so")


def build(verbose: bool = False) -> str:
    """Compiles the sources side by side, every one of them every time, and links them."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as work, ThreadPoolExecutor(4) as pool:
        objects = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        list(pool.map(lambda so: _hipcc(["-c", so[0], "-o", so[1]], verbose), zip(SOURCES, objects)))
        _hipcc(["-shared", *objects, "-o", tmp], verbose)
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
        any(os.path.getmtime(p) > os.path.getmtime(ARGS_LIB) for p in [ARGS_SOURCE, *PUBLIC_HEADERS])


if __name__ == "__main__":
    print(build(verbose=True))
