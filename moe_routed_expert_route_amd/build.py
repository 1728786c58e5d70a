"""Build step: compile the sources in csrc/ for gfx950 into libmoe_route.so next to this file."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
SRCS = [os.path.join(HERE, "csrc", f) for f in ("moe_route.hip", "moe_ops.hip")]
LIB = os.path.join(HERE, "libmoe_route.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # no packed-FP32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # IEEE float32 exactly as written: no FMA contraction, correctly rounded division, denormals
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    # leading scalar kernel arguments arrive preloaded in scalar registers (gfx950)
    "-mllvm", "-amdgpu-kernarg-preload-count=8",
]


def _run(cmd) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stderr[-4000:])
    return res.stderr


def build(verbose: bool = False) -> str:
    """Always recompiles (the sources side by side), in a folder of its own; replaces the library atomically."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    with tempfile.TemporaryDirectory(prefix="build.", dir=os.path.dirname(LIB)) as work:
        objs = [os.path.join(work, os.path.splitext(os.path.basename(s))[0] + ".o") for s in SRCS]
        with ThreadPoolExecutor(len(SRCS)) as pool:
            logs = list(pool.map(lambda so: _run([hipcc, *HIPCC_FLAGS, "-c", "-o", so[1], so[0]]), zip(SRCS, objs)))
        tmp = os.path.join(work, os.path.basename(LIB))
        logs.append(_run([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp, *objs]))
        os.replace(tmp, LIB)
    if verbose:
        print("".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
