"""Builds libqsgd.so (gfx950) in-tree with hipcc.

Flags: -ffp-contract=off keeps every floating-point expression one IEEE op at a
time (the quantizer's decisions must be reproducible bit for bit); packed fp32
instructions are disabled; denormals are kept (no flush-to-zero).
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libqsgd.so")
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("qsgd_api.hip", "int8_api.hip", "distill_api.hip")]
ARCH = os.environ.get("QSGD_OFFLOAD_ARCH", "gfx950")


OBJECTS = os.path.join(HERE, "_build")

FLAGS = [
    "-O3", "-std=c++17", f"--offload-arch={ARCH}",
    "-fPIC", "-ffp-contract=off", "-fno-fast-math", "-fno-strict-aliasing",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wshadow", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
]


def compile_command(source: str, obj: str, extra=()):
    return ["/opt/rocm/bin/hipcc", *FLAGS, *extra, "-c", source, "-o", obj]


def build(verbose: bool = False) -> str:
    """Compiles the sources side by side, then links them."""
    os.makedirs(OBJECTS, exist_ok=True)
    tmp = LIB + ".tmp"
    objs = [os.path.join(OBJECTS, os.path.basename(s) + ".o") for s in SOURCES]
    running = []
    for src, obj in zip(SOURCES, objs):
        cmd = compile_command(src, obj)
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append((cmd, subprocess.Popen(cmd)))
    failed = [(cmd, p.returncode) for cmd, p in running if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(failed[0][1], failed[0][0])
    subprocess.run(["/opt/rocm/bin/hipcc", "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
