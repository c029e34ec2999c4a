"""Builds libcdrge.so (the HIP kernels and the C ABI of include/cdrge.h) for gfx950, in-tree."""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libcdrge.so")
ARCH = "gfx950"

SOURCES = ("cdrge.hip", "scan.hip", "adapters.hip", "distill.hip", "delta.hip", "scores.hip", "mx.hip")

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 instructions stay off: plain float code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    return shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compiles the sources of csrc (side by side) into libcdrge.so next to this file and returns its path."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as out:
        objects = [os.path.join(out, src.replace(".hip", ".o")) for src in SOURCES]
        runs = [subprocess.Popen([hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c",
                                  os.path.join(CSRC, src), "-o", obj, *(extra or [])],
                                 stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
                for src, obj in zip(SOURCES, objects)]
        texts = [run.communicate()[0] for run in runs]
        failed = any(run.returncode != 0 for run in runs)
        if not failed:
            link = subprocess.run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objects, "-o", tmp],
                                  capture_output=True, text=True)
            texts.append(link.stdout + link.stderr)
            failed = link.returncode != 0
    if verbose or failed:
        print("".join(texts))
    if failed:
        raise RuntimeError("hipcc failed building libcdrge.so")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
