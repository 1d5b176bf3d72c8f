"""Dense layer and training calls without a GPU: refusals of the C ABI and of
the binding, workspace sizes, the generator's known answers, and the 64-bit
definitions of the gradients against differences."""
import ctypes
import os

import numpy as np
import pytest
import torch

import training_ref as R

P, I, D, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_size_t
OK, EINVAL, EUNSUP = 0, -1, -2
F32, BF16 = 0, 1
A = P(0x10000)      # never dereferenced: every refusal comes before a launch
ODD = P(0x10008)    # not at a multiple of 16 bytes


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_macs_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    L = ctypes.CDLL(build.LIB)
    L.moe_linear_workspace_size.argtypes = [I] * 5
    L.moe_linear_workspace_size.restype = SZ
    L.moe_linear_backward_workspace_size.argtypes = [I] * 5
    L.moe_linear_backward_workspace_size.restype = SZ
    L.moe_balance_workspace_size.restype = SZ
    L.moe_linear.argtypes = [P] * 4 + [I] * 5 + [P, P, P, SZ, P]
    L.moe_linear_backward.argtypes = [P] * 4 + [I] * 5 + [P, P, P, P, SZ, P]
    L.moe_balance_loss.argtypes = [P] * 3 + [I] * 3 + [P] * 5 + [SZ, P]
    L.moe_router_backward.argtypes = [P] * 7 + [I] * 4 + [P, P]
    L.moe_combine_dropout.argtypes = [P] * 4 + [D, P] + [I] * 4 + [P, P]
    L.moe_combine_backward.argtypes = [P] * 4 + [D, P] + [I] * 4 + [P, P, P]
    return L


def _linear(lib, x=A, w=A, bias=None, res=None, T=4, K=64, O=32, act=0, dtype=BF16, z=None, y=A,
            ws=A, size=1 << 40):
    return lib.moe_linear(x, w, bias, res, T, K, O, act, dtype, z, y, ws, size, None)


def _linear_bwd(lib, dy=A, x=A, w=A, z=A, T=4, K=64, O=32, act=2, dtype=BF16, dx=A, dw=A, db=A,
                ws=A, size=1 << 40):
    return lib.moe_linear_backward(dy, x, w, z, T, K, O, act, dtype, dx, dw, db, ws, size, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), EINVAL), (dict(T=(1 << 20) + 1), EINVAL), (dict(K=0), EINVAL),
    (dict(O=0), EINVAL), (dict(K=65544), EINVAL), (dict(O=65544), EINVAL),
    (dict(act=-1), EINVAL), (dict(act=5), EINVAL), (dict(dtype=2), EUNSUP),
    (dict(dtype=7), EUNSUP), (dict(K=60), EUNSUP), (dict(O=36), EUNSUP),
    (dict(K=62, dtype=F32), EUNSUP), (dict(O=30, dtype=F32), EUNSUP),
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(x=ODD), EINVAL), (dict(w=ODD), EINVAL), (dict(y=ODD), EINVAL),
    (dict(bias=ODD), EINVAL), (dict(res=ODD), EINVAL), (dict(z=ODD), EINVAL),
    (dict(ws=ODD), EINVAL), (dict(size=0), EINVAL),
    (dict(T=0, x=None, y=None), OK),
])
def test_linear_refusals(lib, kw, rc):
    assert _linear(lib, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), EINVAL), (dict(K=0), EINVAL), (dict(O=65544), EINVAL), (dict(act=5), EINVAL),
    (dict(dtype=2), EUNSUP), (dict(K=60), EUNSUP), (dict(O=36), EUNSUP),
    (dict(dx=None, dw=None, db=None), EINVAL), (dict(dy=None), EINVAL), (dict(z=None), EINVAL),
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(size=0), EINVAL), (dict(dy=ODD), EINVAL), (dict(dx=ODD), EINVAL), (dict(dw=ODD), EINVAL),
    (dict(db=ODD), EINVAL), (dict(z=ODD), EINVAL),
    (dict(T=0, dy=None, z=None, dw=None, db=None), OK),
])
def test_linear_backward_refusals(lib, kw, rc):
    assert _linear_bwd(lib, **kw) == rc


def test_linear_workspaces(lib):
    f, b = lib.moe_linear_workspace_size, lib.moe_linear_backward_workspace_size
    assert f(128, 2048, 768, 4, BF16) > 0 and f(0, 2048, 768, 4, BF16) > 0
    assert f(-1, 64, 64, 0, BF16) == 0 and f(4, 60, 64, 0, BF16) == 0
    # dz of both halves is held
    assert b(1000, 64, 128, 4, BF16) >= 1000 * 256 * 2
    assert b(1000, 64, 128, 2, F32) >= 1000 * 128 * 4
    assert b(4, 64, 64, 9, BF16) == 0
    # the largest limits do not wrap
    assert b(1 << 20, 65536, 65536, 4, F32) > (1 << 20) * 131072 * 4


def _balance(lib, logits=A, ids=A, mask=None, T=4, N=8, k=2, out=A, lse=A, ws=A, size=1 << 40):
    return lib.moe_balance_loss(logits, ids, mask, T, N, k, out, out, out, lse, ws, size, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=(1 << 20) + 1), dict(N=0), dict(N=1025), dict(k=0), dict(k=9),
    dict(logits=None), dict(ids=None), dict(out=None), dict(lse=None), dict(ws=None),
    dict(size=0), dict(ws=P(0x10004))])
def test_balance_refusals(lib, kw):
    assert _balance(lib, **kw) == EINVAL


def test_router_backward_refusals(lib):
    def call(logits=A, ids=A, lse=A, counts=A, dg=A, T=4, N=8, k=2, dtype=F32, out=A):
        return lib.moe_router_backward(logits, ids, None, lse, counts, A, dg, T, N, k, dtype, out,
                                       None)
    for kw in (dict(T=-1), dict(N=0), dict(N=1025), dict(k=9), dict(logits=None), dict(lse=None),
               dict(counts=None), dict(out=None), dict(ids=None)):
        assert call(**kw) == EINVAL, kw
    assert call(dtype=2) == EUNSUP
    assert call(T=0, logits=None, out=None) == OK
    assert lib.moe_balance_workspace_size(4, 0) == 0
    assert lib.moe_balance_workspace_size(-1, 8) == 0
    assert lib.moe_balance_workspace_size(0, 8) > 0


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(k=1025), EINVAL), (dict(H=0), EINVAL),
    (dict(p=-0.1), EINVAL), (dict(p=1.0), EINVAL), (dict(p=float("nan")), EINVAL),
    (dict(rng=None), EINVAL), (dict(rng=P(0x10004)), EINVAL), (dict(dtype=2), EUNSUP),
    (dict(H=68), EUNSUP), (dict(H=68, dtype=F32), EUNSUP), (dict(rows=None), EINVAL),
    (dict(slot_row=None), EINVAL), (dict(gates=None), EINVAL), (dict(out=None, out2=None), EINVAL),
    (dict(rows=ODD), EINVAL), (dict(dense=ODD), EINVAL), (dict(out=ODD), EINVAL),
    (dict(T=0, rows=None, rng=None), OK)])
def test_combine_refusals(lib, kw, rc):
    a = dict(rows=A, slot_row=A, gates=A, dense=A, p=0.5, rng=A, T=4, k=2, H=64, dtype=BF16,
             out=A, out2=A)
    a.update(kw)
    mid = [a["p"], a["rng"], a["T"], a["k"], a["H"], a["dtype"]]
    assert lib.moe_combine_dropout(a["rows"], a["slot_row"], a["gates"], a["dense"], *mid,
                                   a["out"], None) == rc
    assert lib.moe_combine_backward(a["dense"], a["rows"], a["slot_row"], a["gates"], *mid,
                                    a["out"], a["out2"], None) == rc


def test_no_tokens_with_empty_outputs(lib):
    """An empty tensor has a null address: without tokens, outputs of T rows may
    be null and nothing is asked of them."""
    assert _linear_bwd(lib, T=0, dy=None, x=None, z=None, dx=None, dw=None, db=None, size=0, ws=None) == OK
    assert lib.moe_combine_backward(None, None, None, None, 0.0, None, 0, 2, 64, BF16, None, None,
                                    None) == OK
    assert lib.moe_combine_backward(None, None, None, None, 0.5, None, 0, 2, 64, F32, None, None,
                                    None) == OK
    # the other arguments are looked at all the same
    assert _linear_bwd(lib, T=0, K=60, dx=None, dw=None, db=None) == EUNSUP
    assert lib.moe_combine_backward(None, None, None, None, 1.0, None, 0, 2, 64, BF16, None, None,
                                    None) == EINVAL


def test_binding_refuses_host_tensors_and_names():
    from mixture_experts_layer_macs_amd import binding as B
    x, w = torch.zeros(4, 64), torch.zeros(32, 64)
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.moe_linear(x, w, ws)
    with pytest.raises(ValueError, match="activation"):
        B.moe_linear(x, w, ws, act="tanh")
    with pytest.raises(ValueError, match="element type"):
        B.moe_linear(x.half(), w.half(), ws)
    with pytest.raises(ValueError, match="even number"):
        B.moe_linear(x, torch.zeros(33, 64), ws, act="swiglu")
    with pytest.raises(ValueError, match="needs moe_linear's z"):
        B.moe_linear_backward(x, x, w, ws, act="silu", dx=x)
    with pytest.raises(ValueError, match="no gradient"):
        B.moe_linear_backward(x, x, w, ws)
    rows, slot_row, gates = torch.zeros(8, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        B.moe_combine_dropout(rows, slot_row, gates, p=0.1)
    with pytest.raises(ValueError, match="no gradient"):
        B.moe_combine_backward(x, rows, slot_row, gates)
    with pytest.raises(ValueError):
        B.moe_balance_loss(x, slot_row, ws)
    with pytest.raises(ValueError):
        B.moe_router_backward(x, slot_row, torch.zeros(4), torch.zeros(65, dtype=torch.int32))


def test_binding_names_the_input_that_a_gradient_needs():
    from mixture_experts_layer_macs_amd import binding as B
    dy, x, w = torch.zeros(4, 32), torch.zeros(4, 64), torch.zeros(32, 64)
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    with pytest.raises(ValueError, match="dx needs w"):
        B.moe_linear_backward(dy, x, None, ws, dx=x)
    with pytest.raises(ValueError, match="dw needs x"):
        B.moe_linear_backward(dy, None, w, ws, dw=w)
    with pytest.raises(ValueError, match="x or w"):
        B.moe_linear_backward(dy, None, None, ws, dbias=dy[0])
    slot_row, gates = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="d_gates needs out_rows"):
        B.moe_combine_backward(x, None, slot_row, gates, d_gates=gates)
    lse, counts = torch.zeros(4), torch.zeros(65, dtype=torch.int32)
    with pytest.raises(ValueError, match="d_gates needs topk_ids"):
        B.moe_router_backward(x, None, lse, counts, d_gates=gates, k=2)
    with pytest.raises(ValueError, match="k is needed"):
        B.moe_router_backward(x, None, lse, counts)
    with pytest.raises(ValueError, match="2 slots per token"):
        B.moe_router_backward(x, slot_row, lse, counts, k=3)


def test_generator_known_answers():
    """The published test vectors of Philox4x32-10 (zero, all ones, digits of pi)."""
    assert R.philox(0, 0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    ones = (1 << 64) - 1
    assert R.philox(ones, ones, ones) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert R.philox(0x299f31d0a4093822, 0x0370734413198a2e, 0x85a308d3243f6a88) == [
        0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def _quotient(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
def test_linear_gradient_against_differences(act):
    """Central differences in 64 bits: truncation h^2 / 6 |f'''| and rounding
    2^-53 |f| / h stay far below 1e-6 of the sums' scale at h = 1e-5."""
    g = np.random.default_rng(3)
    T, K, O = 5, 8, 6
    W = 2 * O if act == "swiglu" else O
    x, w, b, c = g.normal(size=(T, K)), g.normal(size=(W, K)), g.normal(size=W), g.normal(size=(T, O))
    f = lambda x, w, b: (R.linear(x, w, b, None, act, torch.float32)[0] * c).sum()  # noqa: E731
    z = R.linear(x, w, b, None, act, torch.float32)[1]
    r = R.linear_backward(c, x, w, z, act, torch.float32)
    for name, at, fn in (("dx", x, lambda q: f(q, w, b)), ("dw", w, lambda q: f(x, q, b)),
                         ("db", b, lambda q: f(x, w, q))):
        v = g.normal(size=at.shape)
        scale = np.abs(r[name][0] * v).sum() + 1
        assert abs(_quotient(fn, at, v) - (r[name][0] * v).sum()) < 1e-6 * scale, name


def test_balance_gradient_against_differences():
    g = np.random.default_rng(4)
    T, N, k = 7, 5, 2
    logits = g.normal(size=(T, N))
    logits[2, 1] = -np.inf
    ids = np.stack([g.permutation(N)[:k] for _ in range(T)])
    mask = np.array([1, 1, 1, 0, 1, 1, 1])
    dl, dg = np.array([0.7, 0.3]), g.normal(size=(T, k))

    def f(z):
        r = R.balance(z, ids, mask)
        p = np.exp(z - np.where(mask != 0, r["lse"], 0)[:, None]) * (mask != 0)[:, None]
        return (dl * r["losses"]).sum() + (np.take_along_axis(p, ids, 1) * dg).sum()

    r = R.balance(logits, ids, mask, dl, dg)
    v = g.normal(size=(T, N)) * (mask != 0)[:, None]
    assert abs(_quotient(f, logits, v) - (r["dlogits"] * v).sum()) < 1e-6
    assert (r["dlogits"][3] == 0).all() and r["dlogits"][2, 1] == 0


def test_combine_gradient_against_differences():
    g = np.random.default_rng(5)
    T, k, H = 4, 3, 8
    rows, gates, c = g.normal(size=(T * k, H)), g.random((T, k)), g.normal(size=(T, H))
    slot_row = g.permutation(T * k).reshape(T, k).astype(np.int32)
    slot_row[1] = -1
    slot_row[2, 1] = -1
    m = R.keep(99, 7, T, H, 0.25) / 0.75
    f = lambda rows, gates: (R.combine(rows, slot_row, gates, None, m, torch.float32)[0] * c).sum()  # noqa: E731
    d_rows, _, dg, _ = R.combine_backward(c, rows, slot_row, gates, m, torch.float32)
    v = g.normal(size=rows.shape)
    assert abs(_quotient(lambda q: f(q, gates), rows, v) - np.nansum(d_rows * v)) < 1e-6
    v = g.normal(size=gates.shape)
    assert abs(_quotient(lambda q: f(rows, q), gates, v) - (dg * v).sum()) < 1e-6
