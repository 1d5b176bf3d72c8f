"""Grouped products, norm and gradient clipping without a GPU: refusals of the C
ABI and of the binding, workspace sizes, the clipping table, and the 64-bit
definitions of the gradients against differences."""
import ctypes
import os

import numpy as np
import pytest
import torch

import experts_ref as E

P, I, D, SZ, L64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_size_t, ctypes.c_int64
OK, EINVAL, EUNSUP = 0, -1, -2
F32, BF16 = 0, 1
A = P(0x10000)      # never dereferenced: every refusal comes before a launch
ODD = P(0x10008)    # not at a multiple of 16 bytes
ROWS = 1 << 23


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_macs_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    L = ctypes.CDLL(build.LIB)
    for n in ("moe_grouped_linear_workspace_size", "moe_grouped_linear_backward_workspace_size"):
        getattr(L, n).argtypes, getattr(L, n).restype = [I] * 6, SZ
    L.moe_norm_backward_workspace_size.restype = SZ
    L.moe_grad_clip_workspace_size.argtypes, L.moe_grad_clip_workspace_size.restype = [L64], SZ
    L.moe_grouped_linear.argtypes = [P] * 4 + [I] * 7 + [P, P, P, SZ, P]
    L.moe_grouped_linear_backward.argtypes = [P] * 6 + [I] * 7 + [P, P, P, SZ, P]
    L.moe_norm.argtypes = [P] * 4 + [I] * 3 + [D, I] + [P] * 5
    L.moe_norm_backward.argtypes = [P] * 6 + [I] * 4 + [P] * 4 + [SZ, P]
    L.moe_grad_clip.argtypes = [P, I, L64, D, P, P, SZ, P]
    L.moe_grad_table.argtypes = [P, P, P, P, I, P, P]
    return L


SHARED = [
    (dict(R=-1), EINVAL), (dict(R=ROWS + 1, T=ROWS + 1), EINVAL), (dict(N=0), EINVAL), (dict(N=1025), EINVAL),
    (dict(K=0), EINVAL), (dict(O=0), EINVAL), (dict(K=65544), EINVAL), (dict(O=65544), EINVAL),
    (dict(act=-1), EINVAL), (dict(act=5), EINVAL), (dict(dtype=2), EUNSUP), (dict(K=60), EUNSUP),
    (dict(O=36), EUNSUP), (dict(K=62, dtype=F32), EUNSUP), (dict(T=-1), EINVAL), (dict(T=ROWS + 1), EINVAL),
    (dict(T=0), EINVAL), (dict(token=None, T=5), EINVAL), (dict(T=(1 << 18) + 1, K=4096), EUNSUP),
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(offsets=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(size=0), EINVAL), (dict(x=ODD), EINVAL), (dict(w=ODD), EINVAL), (dict(z=ODD), EINVAL),
    (dict(ws=ODD), EINVAL),
]


@pytest.mark.parametrize("kw,rc", SHARED + [
    (dict(y=None), EINVAL), (dict(y=ODD), EINVAL), (dict(R=0, x=None, y=None, offsets=None), OK)])
def test_grouped_refusals(lib, kw, rc):
    a = dict(x=A, token=A, offsets=A, w=A, T=4, R=8, N=4, K=64, O=32, act=2, dtype=BF16, z=None, y=A, ws=A,
             size=1 << 40)
    a.update(kw)
    assert lib.moe_grouped_linear(*a.values(), None) == rc


@pytest.mark.parametrize("kw,rc", SHARED + [
    (dict(dy=None), EINVAL), (dict(z=None), EINVAL), (dict(dx=None, dw=None), EINVAL), (dict(dy=ODD), EINVAL),
    (dict(dx=ODD), EINVAL), (dict(dw=ODD), EINVAL), (dict(R=0, T=0, dy=None, x=None, z=None, dx=None, dw=None), OK)])
def test_grouped_backward_refusals(lib, kw, rc):
    a = dict(dy=A, x=A, token=A, offsets=A, w=A, z=A, T=4, R=8, N=4, K=64, O=32, act=2, dtype=BF16, dx=A, dw=A,
             ws=A, size=1 << 40)
    a.update(kw)
    assert lib.moe_grouped_linear_backward(*a.values(), None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(R=ROWS, O=8192), EUNSUP), (dict(R=1 << 20, N=1024, O=65536), EUNSUP),
    (dict(R=ROWS, O=16384, act=2), EUNSUP), (dict(R=ROWS, O=8192, ws=None), EINVAL)])
def test_grouped_refuses_more_tiles_than_a_grid_holds(lib, kw, rc):
    """Outputs of 137 GB and more, of sizes that are each within their limits."""
    a = dict(x=A, token=A, offsets=A, w=A, T=4, R=8, N=1, K=8, O=32, act=4, dtype=BF16, z=None, y=A, ws=A, size=1 << 40)
    a.update(kw)
    assert lib.moe_grouped_linear(*a.values(), None) == rc


def test_grouped_workspaces(lib):
    f, b = lib.moe_grouped_linear_workspace_size, lib.moe_grouped_linear_backward_workspace_size
    assert f(64, 8, 64, 64, 0, BF16) > 0 and f(0, 8, 64, 64, 0, BF16) > 0
    assert f(-1, 8, 64, 64, 0, BF16) == 0 and f(4, 0, 64, 64, 0, BF16) == 0 and f(4, 8, 60, 64, 0, BF16) == 0
    assert b(1000, 8, 64, 128, 4, BF16) >= 1000 * 256 * 2  # dz of both halves is held
    assert b(1000, 8, 64, 128, 2, F32) >= 1000 * 128 * 4
    assert b(ROWS, 1024, 65536, 65536, 4, F32) > ROWS * 131072 * 4  # the largest limits do not wrap


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), EINVAL), (dict(T=(1 << 20) + 1), EINVAL), (dict(H=0), EINVAL), (dict(H=65544), EINVAL),
    (dict(kind=2), EINVAL), (dict(kind=-1), EINVAL), (dict(dtype=2), EUNSUP), (dict(H=60), EUNSUP),
    (dict(H=62, dtype=F32), EUNSUP), (dict(eps=-1e-9), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None), EINVAL),
    (dict(sum=None), EINVAL), (dict(sum=A), EINVAL), (dict(x=ODD), EINVAL), (dict(res=ODD), EINVAL), (dict(w=ODD), EINVAL),
    (dict(b=ODD), EINVAL), (dict(sum=ODD), EINVAL), (dict(y=ODD), EINVAL), (dict(T=0, x=None, y=None), OK)])
def test_norm_refusals(lib, kw, rc):
    a = dict(x=A, res=A, w=A, b=A, T=4, H=64, kind=0, eps=1e-5, dtype=BF16, sum=P(0x20000), y=A, mean=None, rstd=None)
    a.update(kw)
    assert lib.moe_norm(*a.values(), None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), EINVAL), (dict(H=65544), EINVAL), (dict(kind=2), EINVAL), (dict(dtype=2), EUNSUP),
    (dict(H=60), EUNSUP), (dict(dy=None), EINVAL), (dict(s=None), EINVAL), (dict(w=None), EINVAL),
    (dict(mean=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dx=None, dw=None, db=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(size=0), EINVAL), (dict(dy=ODD), EINVAL), (dict(s=ODD), EINVAL),
    (dict(dsum=ODD), EINVAL), (dict(dx=ODD), EINVAL), (dict(dw=ODD), EINVAL), (dict(db=ODD), EINVAL),
    (dict(ws=ODD), EINVAL), (dict(T=0, dy=None, s=None, dx=None, dw=None, db=None, ws=None), OK)])
def test_norm_backward_refusals(lib, kw, rc):
    a = dict(dy=A, s=A, w=A, mean=A, rstd=A, dsum=None, T=4, H=64, kind=0, dtype=BF16, dx=A, dw=A, db=A, ws=A,
             size=1 << 40)
    a.update(kw)
    assert lib.moe_norm_backward(*a.values(), None) == rc
    f = lib.moe_norm_backward_workspace_size
    assert f(4, 64, BF16) > 0 and f(0, 64, BF16) > 0 and f(4, 60, BF16) == 0 and f(-1, 64, BF16) == 0


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=(1 << 20) + 1), dict(blocks=-1), dict(max_norm=0.0), dict(max_norm=-1.0),
    dict(max_norm=float("nan")), dict(norm=None), dict(table=None), dict(ws=None), dict(ws=ODD), dict(size=0),
    dict(n=0, blocks=1), dict(table=P(0x10004))])
def test_clip_refusals(lib, kw):
    a = dict(table=A, n=2, blocks=3, max_norm=1.0, norm=A, ws=A, size=1 << 20)
    a.update(kw)
    assert lib.moe_grad_clip(*a.values(), None) == EINVAL
    assert lib.moe_grad_clip_workspace_size(-1) == 0 and lib.moe_grad_clip_workspace_size(0) > 0


def _table(lib, grads, outs, counts, types):
    n = len(grads)
    table, blocks = (L64 * (4 * (n + 1)))(), L64(-1)
    rc = lib.moe_grad_table((P * n)(*grads), (P * n)(*outs), (L64 * n)(*counts), (ctypes.c_int32 * n)(*types), n,
                            table, ctypes.byref(blocks))
    return rc, list(table), blocks.value


def test_clip_table(lib):
    """Blocks of 16 KB from the address rounded down to 16 bytes; empty tensors have none."""
    a, b, c = 0x100000, 0x900002, 0xF00000
    rc, t, blocks = _table(lib, [a, b, None, c], [a, b + 0x100000, None, c], [8193, 8192, 0, 1], [F32, BF16, F32, BF16])
    assert rc == OK
    assert t[0:4] == [a, a, 0 * 2 + 0, 8193] and t[4:8] == [b, b + 0x100000, 3 * 2 + 1, 8192]
    assert t[8:12] == [0, 0, 5 * 2, 0] and t[12:16] == [c, c, 5 * 2 + 1, 1]
    assert t[16:20] == [0, 0, 6 * 2, 0] and blocks == 6


@pytest.mark.parametrize("grads,outs,counts,types,rc", [
    ([0x1000], [0x1000], [8], [2], EUNSUP),
    ([0x1000], [0x1000], [-1], [F32], EINVAL),
    ([None], [0x1000], [8], [F32], EINVAL), ([0x1000], [None], [8], [F32], EINVAL),
    ([0x1002], [0x1002], [8], [F32], EINVAL), ([0x1001], [0x1001], [8], [BF16], EINVAL),
    ([0x1000], [0x2004], [8], [F32], EINVAL),                              # other places modulo 16
    ([0x1000], [0x1010], [8], [F32], EINVAL),                              # into itself
    ([0x1000, 0x1000], [0x1000, 0x1000], [8, 8], [F32, F32], EINVAL),      # the same tensor twice
    ([0x1000, 0x2000], [0x3000, 0x3010], [8, 8], [F32, F32], EINVAL),      # outputs overlap
    ([0x1000, 0x2000], [0x2000, 0x3000], [8, 8], [F32, F32], EINVAL),      # an output over another gradient
    ([0x1000, 0x1020], [0x1000, 0x1020], [8, 8], [F32, F32], OK),          # side by side
    ([0x1000, 0x1000], [0x2000, 0x3000], [8, 8], [F32, F32], OK),          # read twice, written apart
    ([], [], [], [], OK)])
def test_clip_table_refusals(lib, grads, outs, counts, types, rc):
    assert _table(lib, grads, outs, counts, types)[0] == rc


def test_binding_refusals():
    from mixture_experts_layer_macs_amd import binding as B
    x, w, off = torch.zeros(4, 64), torch.zeros(2, 32, 64), torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.moe_grouped_linear(x, w, off, ws)
    with pytest.raises(ValueError, match="activation"):
        B.moe_grouped_linear(x, w, off, ws, act="tanh")
    with pytest.raises(ValueError, match="even number"):
        B.moe_grouped_linear(x, torch.zeros(2, 33, 64), off, ws, act="swiglu")
    with pytest.raises(ValueError, match="no gradient"):
        B.moe_grouped_linear_backward(x, x, w, off, ws)
    with pytest.raises(ValueError, match="dx needs w"):
        B.moe_grouped_linear_backward(x, x, None, off, ws, dx=x)
    with pytest.raises(ValueError, match="dw needs x"):
        B.moe_grouped_linear_backward(x, None, w, off, ws, dw=w)
    with pytest.raises(ValueError, match="needs moe_grouped_linear's z"):
        B.moe_grouped_linear_backward(x, x, w, off, ws, act="silu", dx=x)
    with pytest.raises(ValueError, match="unknown norm"):
        B.moe_norm(x, x[0], kind="batch")
    with pytest.raises(ValueError, match="needs total"):
        B.moe_norm(x, x[0], residual=x)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.moe_norm(x, x[0])
    with pytest.raises(ValueError, match="no gradient"):
        B.moe_norm_backward(x, x, x[0], x[:, 0], ws)
    with pytest.raises(ValueError, match="dx needs weight"):
        B.moe_norm_backward(x, x, None, x[:, 0], ws, dx=x)
    with pytest.raises(ValueError, match="needs mean"):
        B.moe_norm_backward(x, x, x[0], x[:, 0], ws, dx=x)
    with pytest.raises(ValueError, match="no gradients"):
        B.GradList([])
    with pytest.raises(ValueError, match="GPU tensor"):
        B.GradList([x])
    with pytest.raises(ValueError, match="outputs"):
        B.GradList([x], [])
    with pytest.raises(TypeError, match="GradList"):
        B.moe_grad_clip([x], 1.0, ws)


# ----------------------------------------------------- definitions, in 64 bits
def _quotient(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
def test_grouped_gradient_against_differences(act):
    g = np.random.default_rng(3)
    T, N, K, O = 4, 3, 8, 6
    W = 2 * O if act == "swiglu" else O
    token, offsets = np.array([2, 0, 3, 1, 2, 0]), [0, 2, 2, 5]  # the last row belongs to no expert
    x, w, c = g.normal(size=(T, K)), g.normal(size=(N, W, K)), g.normal(size=(6, O))
    f = lambda x, w: (E.grouped(x, token, offsets, w, act, torch.float32)[0] * c[:5]).sum()  # noqa: E731
    z = E.grouped(x, token, offsets, w, act, torch.float32)[1]
    r = E.grouped_backward(c, x, token, offsets, w, z, act, torch.float32)
    v = g.normal(size=w.shape)
    assert abs(_quotient(lambda q: f(x, q), w, v) - (r["dw"][0] * v).sum()) < 1e-6 * np.abs(r["dw"][0] * v).sum()
    v = g.normal(size=x.shape)
    dx = np.zeros_like(x)
    np.add.at(dx, token[:5], r["dx"][0])
    assert abs(_quotient(lambda q: f(q, w), x, v) - (dx * v).sum()) < 1e-6 * (np.abs(dx * v).sum() + 1)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_against_differences(kind):
    g = np.random.default_rng(4)
    T, H, eps = 5, 12, 1e-3
    s, w, b, c, ds = g.normal(size=(T, H)), g.normal(size=H), g.normal(size=H), g.normal(size=(T, H)), g.normal(size=(T, H))
    f = lambda s, w, b: (E.norm(s, w, b, kind, eps, torch.float32)["y"][0] * c).sum() + (s * ds).sum()  # noqa: E731
    st = E.norm(s, w, b, kind, eps, torch.float32)
    r = E.norm_backward(c, s, w, st["mean"][0], st["rstd"][0], ds, kind, torch.float32)
    for name, at, fn in (("dx", s, lambda q: f(q, w, b)), ("dw", w, lambda q: f(s, q, b)), ("db", b, lambda q: f(s, w, q))):
        v = g.normal(size=at.shape)
        assert abs(_quotient(fn, at, v) - (r[name][0] * v).sum()) < 1e-6 * (np.abs(r[name][0] * v).sum() + 1), name


def test_clip_definition():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    assert E.clip(g, 1.0) == (5.0, 0.2) and E.clip(g, 5.0) == (5.0, 1.0) and E.clip([np.array([np.inf])], 1.0)[1] == 1.0
