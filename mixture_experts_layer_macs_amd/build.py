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
           "combine_train.hip", "grouped.hip", "norm.hip", "grad_clip.hip"]
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
COUNTED = {"linear.hip": "mma_", "grouped.hip": "mma_"}

# Sources whose kernels load straight to LDS through inline assembly (dma.h).
DIRECT = ("ffn.hip", "router.hip", "similarity.hip", "linear.hip", "grouped.hip")


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


def _scalars(operand: str) -> set:
    if operand == "m0":
        return {"m0"}
    m = re.fullmatch(r"s(?:(\d+)|\[(\d+):(\d+)\])", operand)
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def _writes(op: str, args: list) -> tuple:
    """The scalar registers whose writing by this instruction a load has to keep
    a distance from, and that distance in wait states."""
    if op.startswith(("v_readfirstlane", "v_readlane")):
        return _scalars(args[0]), 5
    if op.startswith(("v_cmp", "v_div_scale", "v_mad_u64", "v_mad_i64")) or "_co_" in op:
        return set().union(*(_scalars(a) for a in args[:2])), 5
    if op.startswith("s_") and args[0] == "m0" and not op.startswith(("s_cmp", "s_bitcmp")):
        return {"m0"}, 1
    return set(), 0


def _check_hazards(src: str, assembly: str) -> None:
    """The direct-to-LDS loads are inline assembly, for which the compiler does
    not keep the wait states that it keeps before its own: five between a vector
    instruction that writes a scalar register and a load that reads it, one
    between a scalar instruction that writes M0 and the load, which takes its LDS
    address from there.  A load closer than that, on any way that leads to it, may
    use a stale address."""
    kernel, code, labels, jumps = "", [], {}, []  # code: kernel, operation, arguments, text
    for line in assembly.splitlines():
        name = re.match(r"([\w.$]+):", line)
        if name and name[1].startswith("_Z"):
            kernel = name[1]
        text = line.split(";")[0].strip()
        if name:
            labels.setdefault(name[1], []).append(len(code))
        elif text and not text.startswith("."):
            op, _, rest = text.partition(" ")
            args = [a.strip() for a in rest.split(",")]
            if op == "s_branch" or op.startswith("s_cbranch"):
                jumps.append((len(code), args[0]))
            code.append((kernel, op, args, text))
    sources = {}  # jumps that lead to an instruction
    for at, label in jumps:
        for to in labels.get(label, []):
            sources.setdefault(to, []).append(at)
    ends = ("s_branch", "s_endpgm", "s_setpc", "s_trap")
    loads = 0
    for i, (kernel, op, args, text) in enumerate(code):
        if not (op.startswith("buffer_load") and text.endswith(" lds")):
            continue
        loads += 1
        used = set().union(*(_scalars(w) for a in args for w in a.split())) | {"m0"}
        ways, seen = [(i, 0)], set()  # an instruction, wait states between it and the load
        while ways:
            at, away = ways.pop()
            before = list(sources.get(at, []))
            if at > 0 and code[at - 1][0] == kernel and not code[at - 1][1].startswith(ends):
                before.append(at - 1)
            for j in before:
                _, o, a, what = code[j]
                wrote, needs = _writes(o, a)
                if away < needs and wrote & used:
                    raise RuntimeError(f"{src}: {kernel}: {text!r} reads what {what!r} writes {away} wait "
                                       "states before it")
                to = (j, away + (int(a[0], 0) + 1 if o == "s_nop" else 1))
                if to[1] < 5 and to not in seen:
                    seen.add(to)
                    ways.append(to)
    if not loads:
        raise RuntimeError(f"{src}: no direct-to-LDS load in its assembly, so their hazards are not known")


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".hip", ".o"))
        report = ["-Rpass-analysis=kernel-resource-usage"] if src in COUNTED else []
        if src in DIRECT:
            report.append("-save-temps=obj")
        cmd = [cc, *_flags(src), *report, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
        if src in COUNTED:
            _check_scratch(src, r.stderr)
        if src in DIRECT:
            stem = src.replace(".hip", "-hip-")
            with open(os.path.join(BUILD, f"{stem}amdgcn-amd-amdhsa-{ARCH}.s")) as f:
                assembly = f.read()
            for name in os.listdir(BUILD):  # the other intermediate files with it
                if name.startswith((stem, src.replace(".hip", "-host-"), src + "-")):
                    os.remove(os.path.join(BUILD, name))
            _check_hazards(src, assembly)
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
