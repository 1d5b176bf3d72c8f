"""The sizes of the GPU tests reach every kernel of the dense layer that a call
can reach, by the choice that csrc/linear_plan.h makes on 256 compute units."""
import random

import pytest
import torch

import linear_plan as P
import test_gpu_training as G

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    return P.load(str(tmp_path_factory.mktemp("plan")))


def _every_forward():
    cut = [f"{t}{s}" for t in P.TILES for s in ("", " split")] + [f"skinny {n}" for n in (1, 2, 4, 8)]
    f32 = ["32x32", "64x64", "64x64 split", "128x128", "128x128 split"]
    return {f"{k}{g}" for k in [f"bf16 {c}" for c in cut] + [f"f32 {c}" for c in f32] for g in ("", " glu")}


def _every_backward():
    cut = {f"bf16 {d} {t}{s}" for d in ("dx", "dw") for t in P.TILES for s in ("", " split")}
    f32 = {f"f32 {d} {t}" for d in ("dx", "dw")
           for t in ("32x32", "64x64", "64x64 split", "128x128", "128x128 split")}
    return cut | f32 | {"f32 pair", "bf16 pair", "bf16 pair dx split", "bf16 pair dw split", "bf16 pair dx dw split"}


def _small(m, w, k, dtype):
    return dtype == BF16 or m * w * k <= 1 << 34


def test_gpu_tests_reach_every_forward_kernel(plan):
    few = next(m.args[1] for m in G.test_linear_few_tokens_wide_weights.pytestmark if m.args[0] == "T,K,O")
    cases = G.VARIANTS + [(*c, act, BF16) for c in few for act in ("none", "swiglu")]
    for dtype in (BF16, F32):
        for i, (T, K, O) in enumerate(G.LINEAR):
            cases += [(T, K, O, G.ACTS[(i + 3 * j) % 5], dtype) for j in range(2)]
        for m, w, k in G.LARGE:
            if _small(m, w, k, dtype):
                cases += [(m, k, w, "silu", dtype), (m, k, w // 16 * 8, "swiglu", dtype)]
    assert {P.forward(plan, *c) for c in cases} == _every_forward()


def test_gpu_tests_reach_every_backward_kernel(plan):
    cases = list(G.BACK_VARIANTS)
    for dtype in (BF16, F32):
        for i, (T, K, O) in enumerate(G.BACK):
            cases += [(T, K, O, G.ACTS[(i + 2 * j) % 5], dtype) for j in range(2)]
        for m, w, k in G.LARGE:
            if _small(m, w, k, dtype):
                cases += [(m, w, k, "none", dtype), (k, w, m // 8 * 8, "silu", dtype)]
    assert set().union(*(P.backward(plan, *c) for c in cases)) == _every_backward()


def test_no_call_reaches_another_kernel(plan):
    """Sizes over the whole range of the limits, drawn over their logarithm."""
    r = random.Random(7)
    every_f, every_b = _every_forward(), _every_backward()
    for _ in range(20000):
        dtype = r.choice([BF16, F32])
        T, K, O = (int(2 ** r.uniform(0, 20)), int(2 ** r.uniform(3, 16)) // 8 * 8, int(2 ** r.uniform(3, 16)) // 8 * 8)
        act = r.choice(["gelu", "swiglu"])
        assert P.forward(plan, T, K, O, act, dtype) in every_f
        assert P.backward(plan, T, K, O, act, dtype) <= every_b


def test_the_header_is_what_the_library_asks(plan):
    """The workspace sizes of the built library are this header's (without a GPU
    it takes 256 compute units)."""
    from mixture_experts_layer_macs_amd import binding as B
    if torch.cuda.is_available():
        pytest.skip("the card's own number of compute units")
    for T, K, O, act, dtype in G.VARIANTS + G.BACK_VARIANTS + [(0, 64, 64, "none", F32), (5000, 4096, 264, "silu", BF16)]:
        v = (T, K, O, P.ACTS[act], 1 if dtype == BF16 else 0, P.CUS)
        assert B.moe_linear_workspace_size(T, K, O, act, dtype) == plan.forward_bytes(*v)
        assert B.moe_linear_backward_workspace_size(T, K, O, act, dtype) == plan.backward_bytes(*v)
