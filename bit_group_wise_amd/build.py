"""Build libq4.so (the HIP kernels and the C ABI) in-tree for gfx950.

Usage: python -m bit_group_wise_amd.build   (or __graft_entry__.build()).
Compiles every HIP source under csrc/ with hipcc, side by side; the linked
result lands next to this file, where the binding loads it.
"""

from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libq4.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++20",
    "-fPIC",
    # IEEE arithmetic everywhere: no contraction of a*b+c unless written as
    # an explicit fma, no fast-math, denormals kept, correctly rounded
    # binary32 division (the hipcc default, stated here for the reader).
    "-ffp-contract=off",
    "-fno-fast-math",
    "-fno-gpu-flush-denormals-to-zero",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    # no packed fp32 instructions (v_pk_{add,mul,fma}_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def build(verbose: bool = False) -> str:
    """Compile the sources, each on its own and several at a time, and link them."""
    def compile_one(src: str, obj: str) -> None:
        cmd = [HIPCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        pairs = [(s, os.path.join(d, os.path.basename(s) + ".o")) for s in sources()]
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda p: compile_one(*p), pairs))
        subprocess.run([HIPCC, FLAGS[0], "-fPIC", "-shared", *(o for _, o in pairs), "-o", tmp], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB)
