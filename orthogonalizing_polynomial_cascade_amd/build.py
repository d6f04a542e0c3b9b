"""Build libanvil.so in-tree with hipcc for gfx950.

    python -m orthogonalizing_polynomial_cascade_amd.build

Flags: -O3; -ffp-contract=off so every fp32 operation of the elementwise steps rounds on its own
(as the page's separate tensor operations do); packed fp32 instructions disabled for the device
code; correctly rounded fp32 division (hipcc's default) is kept, no fast-math.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libanvil.so")
SOURCES = ["momentum.hip", "gemm.hip", "normalize.hip", "update.hip", "api.hip", "norm.hip",
           "linear.hip", "linear_tiles.hip", "gated.hip", "cross_entropy.hip",
           "cross_entropy_grad.hip", "train_api.hip", "head_api.hip", "adamw.hip",
           "adamw_api.hip"]
ARCH = "gfx950"


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def flags() -> list:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        "-ffp-contract=off",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", os.path.join(ROOT, "include"),
        "-Wall", "-Wno-unused-function",
        # the LDS-DMA inline assembly writes m0, a reserved register the kernels use nowhere else
        "-Wno-inline-asm",
    ]


def build(verbose: bool = False) -> str:
    """Compile every source into libanvil.so (always recompiles).  Returns the library path."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as work:
        def compile_one(source):
            out = os.path.join(work, source + ".o")
            cmd = [hipcc()] + flags() + ["-c", os.path.join(CSRC, source), "-o", out]
            if verbose:
                print(" ".join(cmd), flush=True)
            return out, subprocess.run(cmd, capture_output=True, text=True)

        # the sources are independent of each other: one compiler for each, up to the CPUs given
        jobs = min(len(SOURCES), int(os.environ.get("MAX_JOBS", 0)) or os.cpu_count() or 1, 16)
        with ThreadPoolExecutor(jobs) as pool:
            done = list(pool.map(compile_one, SOURCES))
        _report([r for _, r in done], verbose)
        link = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC"] + [o for o, _ in done] + ["-o", tmp]
        _report([subprocess.run(link, capture_output=True, text=True)], verbose)
    os.replace(tmp, LIB)
    return LIB


def _report(runs, verbose):
    # hipcc's host pass does not know the packed-fp32 feature and says so; that is harmless
    noise = "is not a recognized feature for this target"
    msgs = [l for r in runs for l in (r.stdout + r.stderr).splitlines() if noise not in l and l.strip()]
    if any(r.returncode != 0 for r in runs):
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs))


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
