"""Builds libmoe_dispatch.so (the gfx950 HIP kernels and their C ABI) in-tree with hipcc."""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # keep float arithmetic exactly as written (no contraction of separate multiply/add; every
    # fused multiply-add in the kernels is an explicit fma)
    "-ffp-contract=off",
    # no packed fp32 instructions (v_pk_*_f32) in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def library_path() -> str:
    return os.path.join(HERE, "libmoe_dispatch.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def build(verbose: bool = False) -> str:
    """Compiles the sources side by side (one hipcc each) and links them."""
    out = library_path()
    tmp = out + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)

    with tempfile.TemporaryDirectory() as objects:
        def compile_one(src):
            obj = os.path.join(objects, os.path.basename(src) + ".o")
            run(["hipcc", *HIPCC_FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", "-c", src, "-o", obj])
            return obj

        with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as pool:
            built = list(pool.map(compile_one, sources()))
        run(["hipcc", f"--offload-arch={ARCH}", "-shared", "-fPIC", *built, "-o", tmp])
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
