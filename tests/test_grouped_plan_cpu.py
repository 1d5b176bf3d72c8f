"""The grouped products' choice of kernels (csrc/grouped_plan.h, host code): the
sizes of the GPU tests reach, on a card of 256 compute units, every tile."""
import ctypes
import os
import shutil
import subprocess

import pytest

import experts_cases as C

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_macs_amd", "csrc")
CODE = """
#include "grouped_plan.h"
extern "C" int bf16(int mode, int R, int N, int W, int K) { return moe::grp::tile_choice(mode, R, N, W, K, 256); }
extern "C" int splits(int R, int N, int W, int K) { return moe::grp::split_choice(R, N, W, K, 256); }
extern "C" int f32(int mode, int R, int N, int W, int K) { return moe::grp::tile_choice_f32(mode, R, N, W, K, 256); }
"""
FWD, DX, DW = 0, 1, 2
TILE_256, TILE_128, TILE_128x256, STREAM, SKINNY = range(5)


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    folder = tmp_path_factory.mktemp("plan")
    src, lib = folder / "plan.cpp", folder / "plan.so"
    src.write_text(CODE)
    cc = shutil.which("g++") or shutil.which("c++") or "/opt/rocm/llvm/bin/clang++"
    subprocess.run([cc, "-std=c++17", "-O1", "-fPIC", "-shared", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def _sizes():
    for counts, behind, K, O in C.GROUPS + C.LARGE:
        for W in (O, 2 * O):
            yield sum(counts) + behind, len(counts), W, K


def test_every_bf16_tile_is_tested(plan):
    seen = {(m, plan.bf16(m, *s)) for s in _sizes() if s[0] for m in (FWD, DX, DW)}
    assert seen == {(FWD, TILE_256), (FWD, TILE_128), (FWD, SKINNY), (DX, TILE_256), (DX, TILE_128), (DX, TILE_128x256), (DX, STREAM),
                    (DW, TILE_256), (DW, TILE_128), (DW, STREAM)}


def test_weight_gradients_in_parts_are_tested(plan):
    some = [s for s in _sizes() if s[0] and plan.bf16(DW, *s) == TILE_128 and plan.splits(*s) > 1]
    assert len(some) >= 4 and any(s[1] > 1 for s in some)
    for R, N, W, K in ((64, 1, 128, 128), (8192, 8, 28672, 4096), (300, 8, 64, 64)):
        assert plan.splits(R, N, W, K) == 1


def test_every_fp32_tile_is_tested(plan):
    seen = {(m, plan.f32(m, *s)) for s in _sizes() if s[0] for m in (FWD, DX, DW)}
    assert seen == {(m, e) for m in (FWD, DX, DW) for e in (32, 64, 128)}


def test_no_size_reaches_another_tile(plan):
    for R in (1, 7, 300, 5000, 1 << 17, 1 << 23):
        for N in (1, 8, 63, 64, 512, 513, 1024):
            for W in (8, 128, 136, 1536, 65536, 131072):
                for K in (8, 128, 136, 2048, 65536):
                    assert plan.bf16(FWD, R, N, W, K) in (TILE_256, TILE_128, SKINNY)
                    assert plan.bf16(DX, R, N, W, K) in (TILE_256, TILE_128, TILE_128x256, STREAM)
                    assert plan.bf16(DW, R, N, W, K) in (TILE_256, TILE_128, STREAM)
                    for mode in (DX, DW):
                        assert (plan.bf16(mode, R, N, W, K) == STREAM) <= (64 <= N <= 512)
