"""Build libtg_gemm.so in-tree for gfx950 with hipcc.

Usage: python -m dense_fp16_gemm_02_amd.build  (or call ``build()``).
"""
from __future__ import annotations

from concurrent.futures import ThreadPoolExecutor
import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtg_gemm.so")
ARCH = "gfx950"

SOURCES = [os.path.join(CSRC, "tg_gemm.hip"), os.path.join(CSRC, "tg_ceiling.hip"),
           os.path.join(CSRC, "tg_xent.hip"), os.path.join(CSRC, "tg_ortho.hip"),
           os.path.join(CSRC, "tg_grouped.hip"), os.path.join(CSRC, "tg_embed.hip"),
           os.path.join(CSRC, "tg_adamw.hip"), os.path.join(CSRC, "tile_layout_abi.cpp")]

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++20",
    "-fPIC",
    "-shared",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # the layout checks walk every element of a tile at compile time
    "-fconstexpr-steps=200000000",
    "-Wall",
    "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libtg_gemm.so)")


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile every source, a few at a time, and link them."""
    tmp = LIB + ".tmp"

    def run(*args):
        cmd = [hipcc(), *args]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    with tempfile.TemporaryDirectory() as at, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objects = [os.path.join(at, f"{i}.o") for i in range(len(SOURCES))]
        flags = [f for f in FLAGS if f != "-shared"]
        list(pool.map(lambda so: run(*flags, *extra_flags, f"-I{INCLUDE}", f"-I{CSRC}", "-c", so[0], "-o", so[1]),
                      zip(SOURCES, objects)))
        run(*FLAGS, *extra_flags, *objects, "-o", tmp)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
