"""Every form of the grouped products' kernels on the GPU against the 64-bit
definitions: each size of experts_cases.FORMS with a gated and a plain activation,
rows gathered and not."""
import pytest
import torch

import experts_ref as E
import training_ref as R
from experts_cases import FORM_ACTS, FORMS
from gpu_util import load_binding, needs_gpu
from test_gpu_experts import DTYPES, _grouped_inputs, _guard, _near, _outside, _rand

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def B():
    return load_binding()


@pytest.mark.parametrize("i", range(len(FORMS)))
@pytest.mark.parametrize("act", FORM_ACTS)
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@DTYPES
def test_grouped_forms(B, i, act, gather, dtype):
    print(f"[gpu-test] grouped form {i} {act} {gather} {dtype}", flush=True)
    g, M, rows, O, W, x, w, token, tok, off, offsets = _grouped_inputs(FORMS[i], act, dtype, gather, 200 + i)
    K, N = x.shape[1], len(w)
    ws = B.new_workspace(max(B.moe_grouped_linear_workspace_size(rows, N, K, O, act, dtype),
                             B.moe_grouped_linear_backward_workspace_size(rows, N, K, O, act, dtype)), "cuda")
    ws.fill_(0xFF)
    ybuf, y = _guard((rows, O), dtype)
    zbuf, z = _guard((rows, W), dtype)
    B.moe_grouped_linear(x, w, off, ws, row_token=token, act=act, z=z, y=y)
    x64, w64 = R.f64(x), R.f64(w)
    yr, zr, ey, ez = E.grouped(x64, tok, offsets, w64, act, dtype)
    _near(y[:M], yr, ey, "y")
    _near(z[:M], zr, ez, "z")
    assert _outside(ybuf, M * O) and _outside(zbuf, M * W)
    alone = torch.full_like(y, 7.0)  # without z
    B.moe_grouped_linear(x, w, off, ws, row_token=token, act=act, y=alone)
    assert torch.equal(alone, y)
    dy = _rand(g, (rows, O), 0.5, dtype)
    dy[M:], z[M:] = float("nan"), float("nan")
    xbuf, dx = _guard((rows, K), dtype)
    wbuf, dw = _guard(tuple(w.shape), dtype)
    ws.fill_(0xFF)
    B.moe_grouped_linear_backward(dy, x, w, off, ws, row_token=token, z=z, act=act, dx=dx, dw=dw)
    r = E.grouped_backward(R.f64(dy), x64, tok, offsets, w64, R.f64(z), act, dtype)
    _near(dx[:M], *r["dx"], "dx")
    _near(dw, *r["dw"], "dw")
    assert _outside(xbuf, M * K) and _outside(wbuf, dw.numel())
