"""Build libpca_hist.so (HIP, gfx950) in-tree.

Run ``python -m partitioned_chip_accumulation_amd.build`` or call ``build()``.
Every call compiles from source.
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
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libpca_hist.so")
SOURCES = ["hist_api.hip", "hist_bench.hip", "hist_tune.hip", "hist_static.hip",
           "hist_model.hip", "experts_group.hip", "experts_combine.hip", "experts_matmul.hip",
           "experts_dw.hip", "experts_int8.hip"]
JOBS = 6  # compilers at one time

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # packed fp32 instructions stay off
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    errors = [ln for ln in (res.stderr or "").splitlines()
              if "packed-fp32-ops" not in ln]
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(errors))
    if verbose and errors:
        print("\n".join(errors), file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compile every source (several at a time) and link the library."""
    tmp = LIBRARY + ".tmp"
    with tempfile.TemporaryDirectory() as d, ThreadPoolExecutor(JOBS) as pool:
        objects = [os.path.join(d, s + ".o") for s in SOURCES]
        list(pool.map(lambda so: _run(
            [hipcc(), *HIPCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c",
             os.path.join(CSRC, so[0]), "-o", so[1]], verbose), zip(SOURCES, objects)))
        _run([hipcc(), "--offload-arch=gfx950", "-shared", *objects, "-o", tmp], verbose)
    os.replace(tmp, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose=True))
