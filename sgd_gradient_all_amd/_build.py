"""Build libddl.so in-tree with hipcc for gfx950.

Flags: no fast-math, no fp contraction, fp32 denormals kept, HIP's correctly
rounded fp32 division (the default), and packed fp32 instructions disabled.
"""
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libddl.so")
SOURCES = [os.path.join(HERE, "csrc", f)
           for f in ("schedule.cpp", "plan.cpp", "step_kernels.hip", "fused_kernel.hip",
                     "lars_kernels.hip", "linear_kernels.hip",
                     "adamw_kernels.hip", "muon_kernels.hip", "optimizer.cpp",
                     "cross_entropy_loss.hip", "cross_entropy_grad.hip", "adamw8_kernels.hip")]

HIP_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
             "-Wall", "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def build(verbose=False):
    """Every source to an object of its own, side by side, then one library."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, os.path.basename(f) + ".o") for f in SOURCES]

        def compile_one(pair):
            cmd = [hipcc, *HIP_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", pair[0],
                   "-o", pair[1]]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.check_call(cmd)

        with ThreadPoolExecutor(max_workers=8) as pool:
            list(pool.map(compile_one, zip(SOURCES, objects)))
        subprocess.check_call([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", *objects,
                               "-o", LIB + ".tmp"])
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
