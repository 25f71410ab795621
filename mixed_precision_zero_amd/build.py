"""Build libz1.so for gfx950 in-tree with hipcc.

Flags that matter for the results:
  -ffp-contract=off      no fused multiply-add is formed from separate
                         multiplies and adds, so every binary64 operation of
                         the AdamW update rounds where the definition rounds
  (no fast-math)         IEEE division and square root, denormals kept
  -target-feature -packed-fp32-ops
                         no packed two-lane fp32 instructions are generated
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libz1.so")
SOURCES = [os.path.join(CSRC, "z1_api.hip"), os.path.join(CSRC, "z1_kernels.hip"),
           os.path.join(CSRC, "z1_probe.hip"), os.path.join(CSRC, "z1_ops_api.hip"),
           os.path.join(CSRC, "z1_muon.hip"), os.path.join(CSRC, "z1_embed.hip"),
           os.path.join(CSRC, "z1_loss.hip"), os.path.join(CSRC, "z1_layers_api.hip"),
           os.path.join(CSRC, "z1_layers.hip"), os.path.join(CSRC, "z1_linear.hip")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-ffp-contract=off", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I" + INCLUDE, "-I" + CSRC]


def compile_command(source: str, out: str) -> list:
    return [HIPCC, *FLAGS, "-c", "-o", out, source]


def link_command(objects: list, out: str = LIB) -> list:
    return [HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", out, *objects]


def build(out: str = LIB, verbose: bool = False) -> str:
    """Compiles every source, up to eight at a time, and links them."""
    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    with tempfile.TemporaryDirectory() as at:
        objects = [os.path.join(at, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(run, [compile_command(s, o) for s, o in zip(SOURCES, objects)]))
        tmp = out + ".tmp"
        run(link_command(objects, tmp))
    os.replace(tmp, out)   # never leave a half-written library behind
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
