"""Build libepdc.so in-tree with hipcc for gfx950.

Each call compiles every source again (the build check must not trust a
stale library).  Objects go to combine_count_amd/_build/, the library to
combine_count_amd/libepdc.so.
"""
from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libepdc.so")
SOURCES = ["epdc_api.cpp", "epdc_api_ops.cpp", "epdc_api_experts.cpp", "dispatch.hip", "combine.hip", "combine_push.hip",
           "route.hip", "mx.hip", "group.hip", "product.hip", "dense_linear.hip", "dense_linear_int.hip",
           "dense_rows_grad.hip", "dense_weights_grad.hip", "gate.hip", "int8.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

COMMON = [
    "-O3", "-std=c++17", "-fPIC", "-Wall",
    # the only fused multiply-adds are the explicit ones
    "-ffp-contract=off",
]
# device code only: no packed fp32 (v_pk_*_f32) code generation
DEVICE = ["-x", "hip", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    def compile_one(src):
        obj = os.path.join(BUILD, src + ".o")
        cmd = [HIPCC, *(DEVICE if src.endswith(".hip") else []), *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
        return obj, cmd, subprocess.run(cmd, capture_output=True, text=True)

    objs = []
    with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:  # the products' kernels take half a minute a file
        for obj, cmd, r in pool.map(compile_one, sorted(SOURCES, key=lambda s: not s.startswith("dense"))):
            if verbose:
                print(" ".join(cmd), flush=True)
            # hipcc's host pass does not know the device feature flag: drop that note
            noise = "is not a recognized feature for this target"
            msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
            if msg.strip() and (verbose or r.returncode):
                print(msg, flush=True)
            if r.returncode:
                raise subprocess.CalledProcessError(r.returncode, cmd)
            objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
