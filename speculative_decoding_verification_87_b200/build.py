"""Build libspecverify.so (sm_100a) in-tree with nvcc.

    python -m speculative_decoding_verification_87_b200.build [--force]

The library is built from csrc/*.cu (specverify.cu with its headers,
noalloc.cu, walk.cu with sv_walk.cuh, plug.cu, shard.cu, beam.cu, reorder.cu,
weight.cu and evict.cu), compiled for sm_100a only, with static cudart and
-lineinfo.
"""
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libspecverify.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-shared",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "specverify.h")])


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    srcs = _sources()
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(s) for s in srcs)):
        return LIB
    cmd = [NVCC, *NVCC_FLAGS, *extra, "-o", LIB + ".tmp",
           *sorted(glob.glob(os.path.join(CSRC, "*.cu")))]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force="--force" in sys.argv or bool(extra), verbose=True, extra=extra))
