"""Build libmoe_macs.so (gfx950) in-tree with hipcc.

Each HIP source is compiled to an object in parallel, then linked into one
shared library next to this file.  The units that evaluate the
double-precision capacity formula (capacity and fused routing) are compiled
with -ffp-contract=off, so it is evaluated one rounded operation at a time.
Packed fp32 instructions are disabled for all device code.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_macs.so")
SOURCES = ["route.hip", "sere.hip", "capacity.hip", "dispatch.hip",
           "routing_fused.hip", "ffn.hip", "combine.hip", "entropy.hip",
           "router.hip", "similarity.hip", "linear.hip", "balance.hip",
           "combine_train.hip"]
ARCH = os.environ.get("MOE_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc",
                 shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; the MoE library needs ROCm to build")


def _flags(src: str) -> list:
    f = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wno-unused-command-line-argument"]
    if src in ("capacity.hip", "routing_fused.hip"):
        f.append("-ffp-contract=off")
    return f


# Kernels whose loops wait for counted vector-memory instructions: a register
# spilled to scratch memory would add instructions to the count.
COUNTED = {"linear.hip": "mma_"}


def _check_scratch(src: str, remarks: str) -> None:
    found = [(name, size) for name, size in re.findall(
        r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+)", remarks, flags=re.S)
        if COUNTED[src] in name]
    if not found:  # a renamed kernel, or remarks in another form
        raise RuntimeError(f"{src}: the compiler's remarks name no kernel {COUNTED[src]!r}, so its use "
                           "of scratch memory is not known")
    for name, size in found:
        if int(size) != 0:
            raise RuntimeError(f"{src}: {name} uses {size} bytes of scratch memory per lane; its "
                               "counted waits need every value in registers")


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".hip", ".o"))
        report = ["-Rpass-analysis=kernel-resource-usage"] if src in COUNTED else []
        cmd = [cc, *_flags(src), *report, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
        if report:
            _check_scratch(src, r.stderr)
        if verbose and r.stderr.strip():
            print(r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(min(8, len(SOURCES))) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
