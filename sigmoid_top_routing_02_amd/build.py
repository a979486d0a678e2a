"""Builds libmoefp8.so (the HIP kernels + C ABI) for gfx950, in-tree."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoefp8.so")
ROOT = os.path.dirname(HERE)

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-ffp-contract=off",            # every FMA in the kernels is explicit
    "-fno-fast-math",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
    # no wave-level rewriting of atomics: the GEMM's next-tile request must not
    # be waited for (with every DMA in flight) right where it is issued
    "-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
]

# Every source but the MXFP4 product takes MFMA results in VGPRs: the VALU
# consumes every slice there.  That product chains its results through the matrix
# instruction and fills the accumulation registers with them.
VGPR_RESULTS = ["-mllvm", "-amdgpu-mfma-vgpr-form"]
CHAINED = ("mxgemm.hip",)


def flags_of(source):
    return FLAGS + ([] if os.path.basename(source) in CHAINED else VGPR_RESULTS)


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("hipcc failed to build libmoefp8.so")
    # warnings of a build that went through, but for the host pass's remark on a flag for the GPU
    said = [line for line in r.stderr.splitlines(True) if "'-packed-fp32-ops' is not a recognized feature" not in line]
    sys.stderr.write("".join(said))


def build(verbose: bool = False) -> str:
    """Compiles every source to an object, a few at a time, and links them."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as obj:
        def compile_one(src):
            out = os.path.join(obj, os.path.basename(src) + ".o")
            flags = [f for f in flags_of(src) if f != "-shared"]
            _run([HIPCC, *flags, "-I", os.path.join(ROOT, "include"), "-c", "-o", out, src], verbose)
            return out

        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
            objects = list(ex.map(compile_one, sources()))
        _run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp, *objects], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
