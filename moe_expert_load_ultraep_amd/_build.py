"""Build the HIP library in place: ``libultraep.so`` next to this file.

hipcc compiles every source under ``csrc/`` for gfx950.
Packed-fp32 instruction selection is switched off for all device code.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libultraep.so")
SOURCES = ["ultraep_kernels.hip", "ultraep_combine.hip", "ultraep_weights.hip", "ultraep_abi.hip",
           "ultraep_quant.hip", "ultraep_gemm.hip", "ultraep_grads.hip", "ultraep_experts_abi.hip",
           "ultraep_route.hip", "ultraep_norm.hip", "ultraep_glu.hip", "ultraep_layer_abi.hip"]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the ROCm toolchain is required to build libultraep.so")


def command(out: str = LIB) -> list:
    return [hipcc(), "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-function", "-I", INCLUDE, "-I", CSRC,
            *[os.path.join(CSRC, s) for s in SOURCES], "-o", out]


def _run(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")


def build(verbose: bool = False) -> str:
    """Compile the library (always recompiles) and return its path.

    What command() does, each source by a compiler of its own, as many at once as there are CPUs (at most 8)."""
    tmp = LIB + ".tmp"
    flags = [a for a in command(tmp)[:-2] if a != "-shared" and not a.endswith(".hip")]
    with tempfile.TemporaryDirectory() as folder, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objects = [os.path.join(folder, s + ".o") for s in SOURCES]
        jobs = [pool.submit(_run, [*flags, "-c", os.path.join(CSRC, s), "-o", o], verbose) for s, o in zip(SOURCES, objects)]
        for j in jobs:
            j.result()
        _run([hipcc(), "--offload-arch=gfx950", "-fPIC", "-shared", *objects, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
