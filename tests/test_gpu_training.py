"""The dense layer, the router's losses and the training combine on the GPU,
through the binding, against the 64-bit definitions of training_ref."""
import numpy as np
import pytest
import torch
from scipy.special import ndtr

import training_ref as R
from gpu_util import load_binding, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def B():
    return load_binding()


def _rand(g, shape, scale=1.0, dtype=F32):
    return (torch.from_numpy(g.normal(size=shape)) * scale).to(dtype).cuda()


def _near(got, want, bound, what):
    got = R.f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound + 1e-30)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / (bound + 1e-30), 0)), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} over the bound, e.g. at {i}: "
                             f"{got[i]} for {want[i]}, bound {bound[i]:.3e}")


def _guard(shape, dtype, pad=64):
    """A contiguous tensor inside a buffer whose other elements stay as they were."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    return buf, buf[pad:pad + n].view(shape), pad


def _untouched(buf, pad):
    return bool((buf[:pad] == 7).all() and (buf[-pad:] == 7).all())


# --------------------------------------------------------------------- linear
# T, K, O: single tokens, a few rows, sizes around every tile edge, reduction
# lengths that end inside a slice, more columns than a tile
LINEAR = [
    (1, 8, 8), (1, 2048, 1536), (1, 2056, 24), (2, 136, 264), (3, 64, 8), (5, 1032, 72),
    (15, 520, 40), (16, 256, 128), (17, 264, 136), (31, 72, 1000), (33, 2048, 16), (64, 776, 200),
    (65, 4104, 48), (100, 768, 2048), (127, 200, 136), (128, 64, 256), (129, 328, 264),
    (200, 1032, 520), (255, 128, 128), (257, 264, 248), (300, 520, 776), (512, 4096, 64),
    (700, 72, 1544), (1030, 264, 1544), (2100, 136, 264),
]
ACTS = ["none", "relu", "silu", "gelu", "swiglu"]


def _linear_inputs(T, K, O, act, dtype, seed, bias, residual):
    g = np.random.default_rng(seed)
    W = 2 * O if act == "swiglu" else O
    x = _rand(g, (T, K), 1.0, dtype)
    w = _rand(g, (W, K), K ** -0.5, dtype)
    b = _rand(g, (W,), 0.5, dtype) if bias else None
    r = _rand(g, (T, O), 1.0, dtype) if residual else None
    return g, x, w, b, r


@pytest.mark.parametrize("i", range(len(LINEAR)))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear(B, i, dtype):
    T, K, O = LINEAR[i]
    for j in range(2):  # two of the activations with each size, all of them over the sizes
        act = ACTS[(i + 3 * j) % 5]
        bias, residual, keep = (i + j) % 2 == 0, (i + j) % 3 != 0, (i + j) % 4 < 2
        print(f"[gpu-test] linear {T} {K} {O} {act} {dtype}", flush=True)
        g, x, w, b, r = _linear_inputs(T, K, O, act, dtype, 10 * i + j, bias, residual)
        ws = B.new_workspace(B.moe_linear_workspace_size(T, K, O, act, dtype), "cuda")
        ybuf, y, pad = _guard((T, O), dtype)
        zbuf, z, _ = _guard((T, w.shape[0]), dtype)
        B.moe_linear(x, w, ws, bias=b, residual=r, act=act, z=z if keep else None, y=y)
        yr, zr, ey, ez = R.linear(R.f64(x), R.f64(w), R.f64(b), R.f64(r), act, dtype)
        _near(y, yr, ey, "y")
        if keep:
            _near(z, zr, ez, "z")
        assert _untouched(ybuf, pad) and _untouched(zbuf, pad)
        first = y.clone()
        ws.fill_(0xFF)  # the workspace needs no initialisation
        B.moe_linear(x, w, ws, bias=b, residual=r, act=act, z=z if keep else None, y=y)
        assert torch.equal(first, y)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_linear_residual_in_place_and_no_tokens(B, dtype, T):
    g, x, w, b, r = _linear_inputs(T, 136, 264, "gelu", dtype, 5, True, True)
    ws = B.new_workspace(B.moe_linear_workspace_size(T, 136, 264, "gelu", dtype), "cuda")
    want = B.moe_linear(x, w, ws, bias=b, residual=r, act="gelu")
    B.moe_linear(x, w, ws, bias=b, residual=r, act="gelu", y=r)
    assert torch.equal(want, r)
    assert B.moe_linear(x[:0], w, ws, bias=b, act="gelu").shape == (0, 264)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,K,O", [(40, 72, 136), (300, 200, 264), (7, 2056, 40)])
def test_linear_keeps_rows_and_columns_apart(B, dtype, T, K, O):
    """A token of NaN and a weight row of infinities reach only their own
    output row and column; a reduction length inside a slice reads no
    neighbour (the operands are followed by NaN)."""
    g, x, w, b, _ = _linear_inputs(T, K, O, "none", dtype, 6, False, False)
    ws = B.new_workspace(B.moe_linear_workspace_size(T, K, O, "none", dtype), "cuda")
    clean = B.moe_linear(x, w, ws)
    hold = torch.full((2 * (T + O) * K + 512,), float("nan"), dtype=dtype, device="cuda")
    xs, wsx = hold[:T * K].view(T, K), hold[T * K + 256:T * K + 256 + O * K].view(O, K)
    xs.copy_(x)
    wsx.copy_(w)
    assert torch.equal(B.moe_linear(xs, wsx, ws), clean)
    xs[T // 2] = float("nan")
    wsx[O // 3] = float("inf")
    y = B.moe_linear(xs, wsx, ws)
    rows = torch.arange(T, device="cuda") != T // 2
    cols = torch.arange(O, device="cuda") != O // 3
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert y[T // 2].isnan().all() and not y[rows][:, O // 3].isfinite().any()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_activations_at_extreme_values(B, dtype):
    """Large and infinite arguments: the activations' limits, no NaN."""
    v = [0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 100.0, -100.0, 1e4, -1e4, 1e30, -1e30,
         float("inf"), -float("inf")]
    x = torch.zeros(len(v), 8, dtype=dtype, device="cuda")
    x[:, 0] = torch.tensor(v, dtype=dtype)
    w = torch.zeros(16, 8, dtype=dtype, device="cuda")
    w[:, 0] = 1
    ws = B.new_workspace(1 << 16, "cuda")
    z = R.f64(x[:, 0])
    for act, low in (("relu", 0.0), ("silu", None), ("gelu", None)):
        y = R.f64(B.moe_linear(x, w, ws, act=act))
        fin = np.isfinite(z)
        want = R.act_value(z, act)
        assert np.all(np.abs(y[fin] - want[fin][:, None]) <=
                      (2 * R.half(dtype) * np.abs(want) + R.ACT * R.U * (np.abs(z) + 1))[fin][:, None] + 1e-30)
        assert np.all(y[12] == np.inf)


def _act_of(B, z, act, dtype):
    """act(z) of the kernels for a vector z that the type holds: products by 1 and 0."""
    x = torch.zeros(len(z), 8, dtype=dtype, device="cuda")
    x[:, 0] = z
    w = torch.zeros(8, 8, dtype=dtype, device="cuda")
    w[:, 0] = 1
    ws = B.new_workspace(B.moe_linear_workspace_size(len(z), 8, 8, act, dtype), "cuda")
    y = B.moe_linear(x, w, ws, act=act)
    assert (y == y[:, :1]).logical_or(y.isnan()).all()
    return R.f64(y[:, 0])


def _slope_of(B, z, act, dtype):
    """act'(z) of the kernels: the bias gradient of one token with dy = 1."""
    n = len(z)
    one, x = torch.ones(1, n, dtype=dtype, device="cuda"), torch.zeros(1, 8, dtype=dtype, device="cuda")
    ws = B.new_workspace(B.moe_linear_backward_workspace_size(1, 8, n, act, dtype), "cuda")
    db = torch.empty(n, dtype=dtype, device="cuda")
    B.moe_linear_backward(one, x, None, ws, z=z[None].contiguous(), act=act, dbias=db)
    return R.f64(db)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_gelu_is_exact_relative_to_itself(B, dtype):
    """The tail m Phi(-m), m = |z|, is relative to itself.  Roundings in units of
    U = 2^-24: the exponent's m^2/2 three times (1.5 m^2), the exponential 2, the
    argument of the fit 3 times its condition 3.2, its last steps 3 times their
    amplification 2.5, the products 3; 32 in all.  On top of it the fit's own
    error, 5e-6 for bf16 and 6e-8 for fp32, and half a step of the output."""
    z = torch.linspace(-12.5, 12.5, 2000, dtype=torch.float64).to(dtype).cuda()
    zd = R.f64(z)
    rel = (1.5 * zd ** 2 + 32) * R.U + (5e-6 if dtype == BF16 else 6e-8)
    tail, rise = ndtr(-np.abs(zd)), np.abs(zd) * np.exp(-zd ** 2 / 2) / np.sqrt(2 * np.pi)
    want = np.where(zd < 0, zd * tail, zd - zd * tail)
    pos, h = (zd > 0) * 2 * R.U, 1.01 * R.half(dtype)
    _near(torch.from_numpy(_act_of(B, z, "gelu", dtype)), want,
          rel * np.abs(zd) * tail + pos * np.abs(zd) + h * np.abs(want) + 1e-37, "gelu")
    want = np.where(zd < 0, tail - rise, 1 - tail + rise)
    # two terms, of which the second has two more roundings
    _near(torch.from_numpy(_slope_of(B, z, "gelu", dtype)), want,
          (rel + 4 * R.U) * (tail + rise) + pos + h * np.abs(want) + 1e-37, "gelu'")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_activations_reach_their_limits(B, act, dtype):
    """From -100 on the activations and their slopes are 0 (z e^z and z phi(z) lie
    below fp32's range), from 100 on z and 1, infinities included; NaN shows."""
    low = torch.tensor([-100.0, -128.0, -129.0, -1e3, -1e4, -1e30, torch.finfo(dtype).min, -float("inf")], dtype=dtype)
    z = torch.cat([low, -low]).cuda()
    want = torch.cat([torch.zeros_like(low), -low])
    assert np.array_equal(np.abs(_act_of(B, z, act, dtype)), R.f64(want))
    assert np.array_equal(np.abs(_slope_of(B, z, act, dtype)), np.repeat([0.0, 1.0], 8))
    z[3] = z[12] = float("nan")
    nan = np.isin(np.arange(16), [3, 12])
    assert np.array_equal(np.isnan(_act_of(B, z, act, dtype)), nan)
    if act != "relu":  # a unit of NaN passes dy on
        assert np.array_equal(np.isnan(_slope_of(B, z, act, dtype)), nan)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_swiglu_of_closed_and_open_gates(B, dtype):
    """A gate far below 0 closes its column and its gradients, whatever dy is;
    one far above passes the up half; the others do not change."""
    inf, big = float("inf"), torch.finfo(dtype).max
    t = lambda *v: torch.tensor(v, dtype=dtype, device="cuda")  # noqa: E731
    x, w = torch.zeros(1, 8, dtype=dtype, device="cuda"), torch.zeros(16, 8, dtype=dtype, device="cuda")
    x[0, 0] = 1
    w[:8, 0], w[8:, 0] = t(-big, -1e30, -200.0, -1.0, 0.0, 2.0, 200.0, 1e30), 3.0
    ws = B.new_workspace(B.moe_linear_workspace_size(1, 8, 8, "swiglu", dtype), "cuda")
    y, g = R.f64(B.moe_linear(x, w, ws, act="swiglu"))[0], R.f64(w[:8, 0])
    want = 3 * R.act_value(g, "silu")
    assert (y[:3] == 0).all()
    assert np.all(np.abs(y - want) <= 1.01 * R.half(dtype) * np.abs(want) + 3 * R.ACT * R.U * (np.abs(want) + 1))
    z = torch.cat([t(-inf, -1e30, -200.0, -1.0, 0.0, 2.0, 200.0, inf), t(3.0).repeat(8)])[None]
    ws = B.new_workspace(B.moe_linear_backward_workspace_size(1, 8, 8, "swiglu", dtype), "cuda")
    for scale in (1.0, big):
        db = torch.empty(16, dtype=dtype, device="cuda")
        B.moe_linear_backward(t(scale).repeat(8)[None], x, None, ws, z=z, act="swiglu", dbias=db)
        db = R.f64(db)
        assert (db[:3] == 0).all() and (db[8:11] == 0).all()
        if scale == 1:
            assert (db[6:8] == 3).all() and db[14] == 200 and db[15] == np.inf and np.isfinite(db[:15]).all()


BACK = [(1, 64, 72), (2, 2056, 24), (7, 136, 264), (33, 200, 128), (64, 64, 64), (130, 264, 520),
        (251, 136, 264), (256, 512, 256), (300, 1032, 72), (777, 328, 264), (1030, 136, 776),
        (2100, 264, 136), (4100, 64, 40)]


@pytest.mark.parametrize("i", range(len(BACK)))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear_backward(B, i, dtype):
    T, K, O = BACK[i]
    for j in range(2):
        act = ACTS[(i + 2 * j) % 5]
        print(f"[gpu-test] linear backward {T} {K} {O} {act} {dtype}", flush=True)
        g, x, w, b, _ = _linear_inputs(T, K, O, act, dtype, 100 + 10 * i + j, True, False)
        W = w.shape[0]
        dy, z = _rand(g, (T, O), 0.5, dtype), _rand(g, (T, W), 1.0, dtype)
        ws = B.new_workspace(B.moe_linear_backward_workspace_size(T, K, O, act, dtype), "cuda")
        bufs = {"dx": _guard((T, K), dtype), "dw": _guard((W, K), dtype), "db": _guard((W,), dtype)}
        outs = {n: v[1] for n, v in bufs.items()}
        B.moe_linear_backward(dy, x, w, ws, z=z, act=act, dx=outs["dx"], dw=outs["dw"], dbias=outs["db"])
        want = R.linear_backward(R.f64(dy), R.f64(x), R.f64(w), R.f64(z), act, dtype)
        for n, (v, e) in want.items():
            _near(outs[n], v, e, n)
            assert _untouched(bufs[n][0], bufs[n][2]), n
        ws.fill_(0xFF)
        for n in outs:  # each alone gives the same bits
            alone = {m: torch.empty_like(outs[m]) if m == n else None for m in outs}
            B.moe_linear_backward(dy, x, w, ws, z=z, act=act, dx=alone["dx"], dw=alone["dw"],
                                  dbias=alone["db"])
            assert torch.equal(alone[n], outs[n]), n


# Output rows, output columns, reduction: each tile that the products choose on
# 256 compute units, whole and with the reduction split (bf16: 256 x 256, 256 x
# 192, 192 x 256, 128 x 128; fp32: 128 x 128, 64 x 64), with edges inside tiles
# and slices.
LARGE = [(4104, 3080, 512), (2048, 4096, 8192), (3738, 3232, 64), (2304, 2304, 8192),
         (1711, 6952, 64), (1536, 2048, 8192), (144, 64, 856), (8000, 392, 64), (5104, 72, 728),
         (136, 64, 496), (1100, 1544, 264)]


@pytest.mark.parametrize("m,w,k", LARGE)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear_every_tile(B, m, w, k, dtype):
    for act, O in (("silu", w), ("swiglu", w // 16 * 8)):
        if dtype == F32 and m * w * k > 1 << 34:
            continue
        print(f"[gpu-test] linear {m} {k} {O} {act} {dtype}", flush=True)
        g, x, wt, b, r = _linear_inputs(m, k, O, act, dtype, 7, True, True)
        ws = torch.full((B.moe_linear_workspace_size(m, k, O, act, dtype),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        ybuf, y, pad = _guard((m, O), dtype)
        zbuf, z, _ = _guard((m, wt.shape[0]), dtype)
        B.moe_linear(x, wt, ws, bias=b, residual=r, act=act, z=z, y=y)
        yr, zr, ey, ez = R.linear(R.f64(x), R.f64(wt), R.f64(b), R.f64(r), act, dtype)
        _near(z, zr, ez, "z")
        _near(y, yr, ey, "y")
        assert _untouched(ybuf, pad) and _untouched(zbuf, pad)


@pytest.mark.parametrize("m,w,k", LARGE)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear_backward_every_tile(B, m, w, k, dtype):
    """T, O chosen so that dx (first) and dw (second) have these sizes."""
    for T, O, act in ((m, k, "none"), (k, m // 8 * 8, "silu")):
        if dtype == F32 and m * w * k > 1 << 34:
            continue
        print(f"[gpu-test] linear backward {T} {w} {O} {act} {dtype}", flush=True)
        g, x, wt, _, _ = _linear_inputs(T, w, O, act, dtype, 8, False, False)
        dy, z = _rand(g, (T, O), 0.5, dtype), _rand(g, (T, O), 1.0, dtype)
        ws = torch.full((B.moe_linear_backward_workspace_size(T, w, O, act, dtype),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        bufs = {"dx": _guard((T, w), dtype), "dw": _guard((O, w), dtype), "db": _guard((O,), dtype)}
        B.moe_linear_backward(dy, x, wt, ws, z=z, act=act, dx=bufs["dx"][1], dw=bufs["dw"][1],
                              dbias=bufs["db"][1])
        want = R.linear_backward(R.f64(dy), R.f64(x), R.f64(wt), R.f64(z), act, dtype)
        for n, (v, e) in want.items():
            _near(bufs[n][1], v, e, n)
            assert _untouched(bufs[n][0], bufs[n][2]), n


@pytest.mark.parametrize("T,K,O", [(1, 14336, 4096), (16, 14336, 4096), (40, 1264, 72), (70, 4096, 512),
                                   (100, 608, 4488), (127, 480, 4264), (128, 4096, 1024)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_few_tokens_wide_weights(B, T, K, O, act):
    g, x, w, b, r = _linear_inputs(T, K, O, act, BF16, 9, True, True)
    ws = torch.full((B.moe_linear_workspace_size(T, K, O, act, BF16),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    ybuf, y, pad = _guard((T, O), BF16)
    B.moe_linear(x, w, ws, bias=b, residual=r, act=act, y=y)
    yr, _, ey, _ = R.linear(R.f64(x), R.f64(w), R.f64(b), R.f64(r), act, BF16)
    _near(y, yr, ey, "y")
    assert _untouched(ybuf, pad)


# Kernels that the sizes above do not reach: the skinny product of gated weights
# for more than 16 tokens, split fp32 tiles, 128 x 128 tiles without a partner,
# both products of a small backward pass split.
VARIANTS = [(29, 944, 2040, "swiglu", BF16), (40, 200, 2920, "swiglu", BF16), (70, 760, 2488, "swiglu", BF16),
            (67, 1124, 3324, "none", F32)]
BACK_VARIANTS = [(154, 49600, 8, "none", BF16), (1, 49592, 72, "swiglu", BF16), (849, 8, 840, "none", BF16),
                 (3143, 304, 1192, "swiglu", BF16)]


@pytest.mark.parametrize("T,K,O,act,dtype", VARIANTS)
def test_linear_other_variants(B, T, K, O, act, dtype):
    g, x, w, b, r = _linear_inputs(T, K, O, act, dtype, 15, True, True)
    ws = torch.full((B.moe_linear_workspace_size(T, K, O, act, dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    (ybuf, y, pad), (zbuf, z, _) = _guard((T, O), dtype), _guard((T, w.shape[0]), dtype)
    B.moe_linear(x, w, ws, bias=b, residual=r, act=act, z=z, y=y)
    yr, zr, ey, ez = R.linear(R.f64(x), R.f64(w), R.f64(b), R.f64(r), act, dtype)
    _near(z, zr, ez, "z")
    _near(y, yr, ey, "y")
    assert _untouched(ybuf, pad) and _untouched(zbuf, pad)


@pytest.mark.parametrize("T,K,O,act,dtype", BACK_VARIANTS)
def test_linear_backward_other_variants(B, T, K, O, act, dtype):
    g, x, w, _, _ = _linear_inputs(T, K, O, act, dtype, 16, False, False)
    W = w.shape[0]
    dy, z = _rand(g, (T, O), 0.5, dtype), _rand(g, (T, W), 1.0, dtype)
    ws = torch.full((B.moe_linear_backward_workspace_size(T, K, O, act, dtype),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    bufs = {"dx": _guard((T, K), dtype), "dw": _guard((W, K), dtype), "db": _guard((W,), dtype)}
    B.moe_linear_backward(dy, x, w, ws, z=z, act=act, dx=bufs["dx"][1], dw=bufs["dw"][1], dbias=bufs["db"][1])
    for n, (v, e) in R.linear_backward(R.f64(dy), R.f64(x), R.f64(w), R.f64(z), act, dtype).items():
        _near(bufs[n][1], v, e, n)
        assert _untouched(bufs[n][0], bufs[n][2]), n


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_relu_shows_nan_and_closes_to_infinity(B, dtype):
    T, K, O = 5, 16, 24
    x = torch.ones(T, K, dtype=dtype, device="cuda")
    w = torch.zeros(O, K, dtype=dtype, device="cuda")
    w[:8, 0], w[8:16, 0] = 2.0, -2.0
    x[3] = float("nan")
    z = torch.empty(T, O, dtype=dtype, device="cuda")
    ws = torch.empty(B.moe_linear_workspace_size(T, K, O, "relu", dtype), dtype=torch.uint8, device="cuda")
    y = B.moe_linear(x, w, ws, act="relu", z=z)
    torch.cuda.synchronize()
    assert y[3].isnan().all() and z[3].isnan().all()
    rows = [0, 1, 2, 4]
    assert (y[rows][:, :8] == 2).all() and (y[rows][:, 8:] == 0).all()
    # dy = inf passes an open unit and is stopped by a closed one
    z[3] = z[2]
    dy = torch.full((T, O), float("inf"), dtype=dtype, device="cuda")
    db = torch.empty(O, dtype=dtype, device="cuda")
    ws = torch.empty(B.moe_linear_backward_workspace_size(T, K, O, "relu", dtype), dtype=torch.uint8,
                     device="cuda")
    B.moe_linear_backward(dy, x, w, ws, z=z, act="relu", dbias=db)
    torch.cuda.synchronize()
    assert (db[:8] == float("inf")).all() and (db[8:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear_backward_without_tokens_writes_zeros(B, dtype):
    x, w = torch.empty(0, 64, dtype=dtype, device="cuda"), torch.ones(48, 64, dtype=dtype, device="cuda")
    dw, db = torch.ones_like(w), torch.ones(48, dtype=dtype, device="cuda")
    ws = B.new_workspace(0, "cuda")
    B.moe_linear_backward(x.new_empty(0, 48), x, w, ws, act="none", dw=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_backward_calls_without_tokens(B, dtype):
    """An empty batch through the binding: each empty gradient alone and all of
    them; the sums over tokens are zeros."""
    e = lambda *s: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    w, ws = torch.ones(48, 64, dtype=dtype, device="cuda"), B.new_workspace(0, "cuda")
    dx, _, _ = B.moe_linear_backward(e(0, 48), e(0, 64), w, ws, dx=e(0, 64))
    assert dx.shape == (0, 64)
    dw, db = torch.ones_like(w), torch.ones(48, dtype=dtype, device="cuda")
    B.moe_linear_backward(e(0, 48), e(0, 64), w, ws, z=e(0, 48), act="gelu", dx=e(0, 64), dw=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()
    S, G = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    for dr, dg in ((e(0, 64), None), (None, torch.empty_like(G)), (e(0, 64), torch.empty_like(G))):
        B.moe_combine_backward(e(0, 64), e(0, 64), S, G, d_out_rows=dr, d_gates=dg)
    assert B.moe_combine_dropout(e(0, 64), S, G, residual=e(0, 64)).shape == (0, 64)
    out = B.moe_balance_loss(torch.empty(0, 16, device="cuda"), S, B.new_workspace(
        B.moe_balance_workspace_size(0, 16), "cuda"))
    assert B.moe_router_backward(torch.empty(0, 16, device="cuda"), S, out["lse"], out["counts"],
                                 d_gates=G, dtype=dtype).shape == (0, 16)


@pytest.mark.parametrize("T,K,O,act", [(1030, 136, 776, "gelu"), (2048, 1024, 384, "swiglu"), (70, 72, 136, "silu")])
def test_linear_backward_rounds_dz_once_and_nothing_else(B, T, K, O, act):
    """dx and dw are the products of dz rounded to bf16: off them by fp32 sums and
    half a step of the result, and by a step of dz where its fp32 value (within e
    of the exact one) may round to either side; the same inputs give the same bits."""
    g, x, w, _, _ = _linear_inputs(T, K, O, act, BF16, 31, False, False)
    W = w.shape[0]
    dy, z = _rand(g, (T, O), 0.5, BF16), _rand(g, (T, W), 1.0, BF16)
    ws = B.new_workspace(B.moe_linear_backward_workspace_size(T, K, O, act, BF16), "cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    B.moe_linear_backward(dy, x, w, ws, z=z, act=act, dx=dx, dw=dw)
    dz, e = R.act_grad(R.f64(dy), R.f64(z), act)
    lo, mid, hi = (R.f64(torch.from_numpy(v).to(BF16)) for v in (dz - e, dz, dz + e))
    step, h = hi - lo, 1.01 * R.half(BF16)
    for got, a, s, b, n in ((dx, mid, step, R.f64(w), W), (dw, mid.T, step.T, R.f64(x), T)):
        v = R.product(a, b)
        err = R.product((n + 2) * R.U * (np.abs(a) + s) + s, np.abs(b))
        _near(got, v, err * (1 + h) + h * np.abs(v), "dx" if got is dx else "dw")
    first = dx.clone(), dw.clone()
    ws.fill_(0xFF)
    B.moe_linear(x, w, ws[:256].new_zeros(B.moe_linear_workspace_size(T, K, O, act, BF16)), act=act)
    B.moe_linear_backward(dy, x, w, ws, z=z, act=act, dx=dx, dw=dw)
    assert torch.equal(first[0], dx) and torch.equal(first[1], dw)


def test_linear_gradient_against_the_kernels_own_differences(B):
    """The fp32 forward kernel's difference quotient along a direction equals
    the 64-bit one up to the forward's rounding over 2h."""
    T, K, O, h = 9, 64, 32, 2.0 ** -6
    for act in ACTS:
        g, x, w, b, _ = _linear_inputs(T, K, O, act, F32, 8, True, False)
        ws = B.new_workspace(1 << 20, "cuda")
        z = torch.empty(T, w.shape[0], device="cuda")
        B.moe_linear(x, w, ws, bias=b, act=act, z=z)
        c = _rand(g, (T, O))
        dx = torch.empty_like(x)
        wsb = B.new_workspace(B.moe_linear_backward_workspace_size(T, K, O, act, F32), "cuda")
        B.moe_linear_backward(c, x, w, wsb, z=z, act=act, dx=dx)
        v = _rand(g, (T, K), 0.1)
        kern, ref, slack = 0.0, 0.0, 0.0
        for sign in (1, -1):
            xs = (x.double() + sign * h * v.double()).float()
            y = B.moe_linear(xs, w, ws, bias=b, act=act)
            yr, _, ey, _ = R.linear(R.f64(xs), R.f64(w), R.f64(b), None, act, F32)
            kern += sign * (R.f64(c) * R.f64(y)).sum() / (2 * h)
            ref += sign * (R.f64(c) * yr).sum() / (2 * h)
            slack += (np.abs(R.f64(c)) * ey).sum() / (2 * h)
        assert abs(kern - ref) <= slack
        # the quotient against the gradient: smooth activations to second order
        # (h |v| ~ 2e-3 relative to unit-scale arguments), relu where no argument changes sign
        if act != "relu":
            dot = (R.f64(dx) * R.f64(v)).sum()
            assert abs(ref - dot) <= 1e-3 * (np.abs(R.f64(dx) * R.f64(v)).sum()) + slack


# -------------------------------------------------------------------- balance
def _balance_inputs(T, N, k, seed, drop=True):
    g = np.random.default_rng(seed)
    logits = (g.normal(size=(T, N)) * 2).astype(np.float32)
    ids = np.stack([g.permutation(N)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    if drop and T:
        ids[g.random((T, k)) < 0.1] = -1
    return g, logits, ids


def _check_balance(B, logits, ids, mask, dl, dg, dtype=F32):
    T, N = logits.shape
    k = ids.shape[1]
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    L, S, M, DL, DG = dev(logits), dev(ids), dev(mask), dev(dl), dev(dg)
    ws = torch.full((max(1, B.moe_balance_workspace_size(T, N)),), 0xFF, dtype=torch.uint8, device="cuda")
    out = B.moe_balance_loss(L, S, ws, token_mask=M)
    buf, dz, pad = _guard((T, N), dtype)
    B.moe_router_backward(L, S, out["lse"], out["counts"], d_losses=DL, token_mask=M, d_gates=DG,
                          dlogits=dz)
    r = R.balance(logits.astype(np.float64), ids, mask, None if dl is None else dl.astype(np.float64),
                  None if dg is None else dg.astype(np.float64))
    assert np.array_equal(out["counts"].cpu().numpy(), r["counts"])
    # fp32 logits up to |z|: exp and log in fp32 (a few units, and |z| 2^-24 from the argument), N-term sums
    zmax = np.abs(logits[np.isfinite(logits)]).max() if np.isfinite(logits).any() else 0.0
    e = (R.ACT + N / 16 + 2 * zmax) * R.U
    fin = np.isfinite(r["lse"])
    got = R.f64(out["lse"])
    assert np.array_equal(got[~fin], r["lse"][~fin])
    _near(torch.from_numpy(got[fin]), r["lse"][fin], e + R.U * np.abs(r["lse"][fin]), "lse")
    _near(out["mean_prob"], r["mean_prob"], 2 * e * r["mean_prob"], "mean_prob")
    zl = np.sqrt(r["losses"][1])
    _near(out["losses"], r["losses"], np.array([2 * e * r["losses"][0], 4 * (e + R.U * zmax) * (zl + 1) * (zl + 1)]),
          "losses")
    # p is off by a relative 2 e (through lse, with |lse| 2^-24 from its own rounding); then N-term sums
    h = R.half(dtype)
    _near(dz, r["dlogits"], 6 * (e + R.U * zmax) * r["scale"] + h * np.abs(r["dlogits"]) * 1.01, "dlogits")
    assert _untouched(buf, pad)
    out2 = B.moe_balance_loss(L, S, ws, token_mask=M)
    for n in out:
        assert torch.equal(out[n], out2[n]), n
    return out, dz


@pytest.mark.parametrize("T,N,k", [(1, 1, 1), (1, 8, 2), (2, 5, 5), (3, 64, 8), (7, 65, 3), (16, 128, 8),
                                   (33, 130, 8), (63, 256, 8), (129, 257, 4), (300, 1000, 8), (40, 1024, 70),
                                   (1500, 31, 2), (5000, 16, 4), (9001, 128, 8)])
def test_balance(B, T, N, k):
    g, logits, ids = _balance_inputs(T, N, k, T + N)
    mask = (g.random(T) > 0.2).astype(np.uint8)
    dl, dg = np.array([0.5, 0.25], np.float32), g.normal(size=(T, k)).astype(np.float32)
    _check_balance(B, logits, ids, mask, dl, dg)
    _check_balance(B, logits, ids, None, dl, None)
    _check_balance(B, logits, ids, None, None, dg, BF16)


def test_balance_masked_places(B):
    """Padding full of NaN and infinities, experts ruled out by -inf, a token
    with nothing left, and a batch of padding alone."""
    g, logits, ids = _balance_inputs(50, 40, 4, 9)
    mask = np.ones(50, np.uint8)
    mask[[0, 7, 49]] = 0
    logits[0] = np.nan
    logits[7] = np.inf
    logits[49, ::2] = -np.inf
    logits[3, 5:] = -np.inf
    logits[4] = -np.inf
    logits[5, :] = -np.inf
    logits[5, 39] = np.finfo(np.float32).min
    logits[6] = np.finfo(np.float32).min
    ids[0] = 1 << 30
    dl, dg = np.array([0.5, 0.25], np.float32), g.normal(size=(50, 4)).astype(np.float32)
    dg[0] = np.nan
    finite = logits.copy()
    # a logsumexp of 3.4e38 squares past fp32: the z loss is left out of this check
    dl[1] = 0
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    L, S, M, DL, DG = (dev(a) for a in (logits, ids, mask, dl, dg))
    ws = B.new_workspace(B.moe_balance_workspace_size(50, 40), "cuda")
    out = B.moe_balance_loss(L, S, ws, token_mask=M)
    dz = R.f64(B.moe_router_backward(L, S, out["lse"], out["counts"], DL, M, DG))
    finite[[0, 7, 49]] = 0
    r = R.balance(finite.astype(np.float64), ids, mask, dl.astype(np.float64),
                  np.nan_to_num(dg.astype(np.float64)))
    assert np.array_equal(out["counts"].cpu().numpy(), r["counts"])
    assert np.allclose(R.f64(out["mean_prob"]), r["mean_prob"], rtol=100 * R.U, atol=0)
    assert abs(float(out["losses"][0]) - r["losses"][0]) <= 100 * R.U * r["losses"][0]
    assert (dz[[0, 4, 7, 49]] == 0).all() and np.isfinite(dz).all()
    assert (dz[3, 5:] == 0).all()
    rows = [t for t in range(50) if t not in (5, 6)]
    assert np.all(np.abs(dz - r["dlogits"])[rows] <= 100 * R.U * r["scale"][rows] + 1e-30)
    M.zero_()
    out = B.moe_balance_loss(L, S, ws, token_mask=M)
    assert all((out[n] == 0).all() for n in out)
    assert (B.moe_router_backward(L, S, out["lse"], out["counts"], DL, M, DG) == 0).all()


@pytest.mark.parametrize("T,N,k", [(9, 5, 2), (9, 64, 4), (1500, 16, 2), (1500, 200, 8)])
def test_balance_shows_a_row_of_nan(B, T, N, k):
    """A kept row of NaN is not a row of -inf: the sums and its gradient say so,
    the other tokens' values do not change."""
    _, logits, ids = _balance_inputs(T, N, k, 5)
    logits, ids = torch.from_numpy(logits).cuda(), torch.from_numpy(ids).cuda()
    ws = torch.empty(B.moe_balance_workspace_size(T, N), dtype=torch.uint8, device="cuda")
    good = B.moe_balance_loss(logits, ids, ws)
    dl = torch.ones(2, device="cuda")
    d0 = B.moe_router_backward(logits, ids, good["lse"], good["counts"], d_losses=dl)
    logits[4] = float("nan")
    bad = B.moe_balance_loss(logits, ids, ws)
    d1 = B.moe_router_backward(logits, ids, bad["lse"], bad["counts"], d_losses=dl)
    torch.cuda.synchronize()
    assert bad["losses"].isnan().all() and bad["mean_prob"].isnan().all() and bad["lse"][4].isnan()
    assert d1[4].isnan().all()
    rest = torch.arange(T, device="cuda") != 4
    assert torch.equal(bad["lse"][rest], good["lse"][rest]) and torch.equal(d1[rest], d0[rest])
    assert torch.equal(bad["counts"], good["counts"])


@pytest.mark.parametrize("T,N,k", [(100, 5, 2), (100, 24, 3), (100, 200, 8), (1500, 31, 2), (1500, 200, 8),
                                   (9001, 120, 4), (20000, 12, 4), (3000, 1000, 8)])
def test_balance_sums_over_tokens_in_64_bits(B, T, N, k):
    """T times the same token: T fp32 values of 24 bits sum exactly in fp64, so
    the means are that token's own probabilities bit for bit; the losses, with
    one more rounding in fp64 each, are off by at most a step."""
    _, logits, ids = _balance_inputs(1, N, k, 3, drop=False)
    one = torch.from_numpy(logits).cuda(), torch.from_numpy(ids).cuda()
    many = tuple(t.repeat(T, 1) for t in one)
    a, b = (B.moe_balance_loss(L, S, B.new_workspace(B.moe_balance_workspace_size(L.shape[0], N), "cuda"))
            for L, S in (one, many))
    assert torch.equal(a["mean_prob"], b["mean_prob"])
    assert (b["lse"] == a["lse"]).all() and torch.equal(b["counts"], a["counts"] * T)
    assert np.all(np.abs(R.f64(a["losses"]) - R.f64(b["losses"])) <= 2 * R.U * R.f64(a["losses"]))


@pytest.mark.parametrize("N", [5, 40, 257])
def test_balance_workspace_at_16_bytes(B, N):
    T, k = 3000, 3
    _, logits, ids = _balance_inputs(T, N, k, 12)
    L, S = torch.from_numpy(logits).cuda(), torch.from_numpy(ids).cuda()
    n = B.moe_balance_workspace_size(T, N)
    a = B.moe_balance_loss(L, S, B.new_workspace(n, "cuda"))
    buf = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    b = B.moe_balance_loss(L, S, buf[16:16 + n])
    assert all(torch.equal(a[m], b[m]) for m in a)
    assert (buf[:16] == 0xFF).all() and (buf[16 + n:] == 0xFF).all()


def test_balance_z_loss_of_large_scores(B):
    """logsumexps of 8e18: the sum of some squares passes fp32's range, their
    mean, 6.4e37, does not."""
    T, N = 100000, 40
    L = torch.full((T, N), 8e18, device="cuda")
    S = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    out = B.moe_balance_loss(L, S, B.new_workspace(B.moe_balance_workspace_size(T, N), "cuda"))
    want = R.f64(L[0, 0]) ** 2  # log 40 is far below a step of 8e18
    assert abs(float(out["losses"][1]) - want) <= R.U * want


@pytest.mark.parametrize("T,N,k", [(9, 5, 2), (40, 16, 4), (40, 30, 3), (300, 64, 8), (65, 130, 8), (33, 300, 8),
                                   (9, 1000, 8)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_router_backward_of_scores_far_from_zero(B, T, N, k, dtype):
    """The gradient depends on differences of scores: a common offset (whose
    logsumexp is rounded to a step of 2^-9) costs nothing.  Differences of scores
    and logsumexp are exact or rounded once, and the exponential's argument once
    more: |z - lse| 2^-23 of each p, a few units of the exponential and the
    reciprocal, N-term sums; dlogits holds three such factors."""
    g, logits, ids = _balance_inputs(T, N, k, 11)
    for offset in (30000.0, -30000.0):
        z = logits + np.float32(offset)
        dg = g.normal(size=(T, k)).astype(np.float32)
        for dl in ((0.5, 0.0), (0.0, 0.25)):  # the z loss's term, 2 lse p / n, is far larger than the other
            dl = np.array(dl, np.float32)
            L, S, DL, DG = (torch.from_numpy(a).cuda() for a in (z, ids, dl, dg))
            out = B.moe_balance_loss(L, S, B.new_workspace(B.moe_balance_workspace_size(T, N), "cuda"))
            dz = B.moe_router_backward(L, S, out["lse"], out["counts"], DL, None, DG, dtype=dtype)
            r = R.balance(z.astype(np.float64), ids, None, dl.astype(np.float64), dg.astype(np.float64))
            span = np.abs(z - r["lse"][:, None]).max()
            e = (R.ACT + N / 16 + 2 * span) * R.U
            _near(dz, r["dlogits"], 6 * e * r["scale"] + 1.01 * R.half(dtype) * np.abs(r["dlogits"]), "dlogits")


def test_router_backward_of_the_lowest_scores(B):
    """A token whose scores are all the type's lowest value is a uniform one."""
    T, N, k = 6, 24, 2
    L = torch.full((T, N), torch.finfo(F32).min, device="cuda")
    S = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    DG = torch.full((T, k), 0.5, device="cuda")
    out = B.moe_balance_loss(L, S, B.new_workspace(B.moe_balance_workspace_size(T, N), "cuda"))
    dz = R.f64(B.moe_router_backward(L, S, out["lse"], out["counts"], d_gates=DG))
    want = np.where(np.arange(N) == 0, (1 - 1 / N) / N, -1 / N / N)  # p_j (u_j - sum p u), u_0 = 1
    assert np.all(np.abs(dz - want) <= 6 * (R.ACT + N / 16) * R.U / N)


def test_balance_without_tokens(B):
    ws = torch.full((B.moe_balance_workspace_size(0, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    out = B.moe_balance_loss(torch.empty(0, 16, device="cuda"),
                             torch.empty(0, 2, dtype=torch.int32, device="cuda"), ws)
    assert all((out[n] == 0).all() for n in out)
    assert out["counts"].shape == (17,)


def test_router_backward_same_expert_twice(B):
    """Gate gradients of one expert named by several slots add up."""
    logits = np.random.default_rng(1).normal(size=(6, 70)).astype(np.float32)
    ids = np.full((6, 3), 66, np.int32)
    ids[:, 2] = 1
    dg = np.arange(18, dtype=np.float32).reshape(6, 3) / 8
    _check_balance(B, logits, ids, None, np.zeros(2, np.float32), dg)


# -------------------------------------------------------------------- combine
def _combine_inputs(T, H, k, dtype, seed):
    g = np.random.default_rng(seed)
    kept = g.random((T, k)) > 0.15
    if T > 2:
        kept[T // 2] = False
    slot_row = np.full((T, k), -1, np.int32)
    slot_row[kept] = g.permutation(int(kept.sum()))
    rows = _rand(g, (T * k, H), 1.0, dtype)
    gates = g.random((T, k)).astype(np.float32)
    return g, rows, slot_row, gates


@pytest.mark.parametrize("T,H,k,p,res", [
    (1, 8, 1, 0.0, False), (1, 2048, 8, 0.1, True), (2, 16, 3, 0.5, True), (3, 264, 8, 0.25, False),
    (5, 1032, 2, 0.1, True), (9, 520, 9, 0.9, True), (17, 64, 20, 0.0, True), (33, 128, 2, 0.1, False),
    (4, 4104, 4, 0.3, True), (70, 40, 5, 0.999999, True)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_combine(B, T, H, k, p, res, dtype):
    g, rows, slot_row, gates = _combine_inputs(T, H, k, dtype, T + H)
    seed, offset = 0x1234_5678_9ABC_DEF0 + T, (1 << 40) + 3
    rng = torch.tensor([seed, offset], dtype=torch.int64, device="cuda") if p else None
    r = _rand(g, (T, H), 1.0, dtype) if res else None
    S, G = torch.from_numpy(slot_row).cuda(), torch.from_numpy(gates).cuda()
    buf, y, pad = _guard((T, H), dtype)
    B.moe_combine_dropout(rows, S, G, p=p, rng=rng, residual=r, y=y)
    m = R.keep(seed, offset, T, H, p) / (1 - p) if p else np.ones((T, H))
    gd = gates.astype(np.float64)
    want, bound = R.combine(R.f64(rows), slot_row, gd, R.f64(r), m, dtype)
    _near(y, want, bound, "y")
    assert _untouched(buf, pad)
    if r is not None:  # in place
        B.moe_combine_dropout(rows, S, G, p=p, rng=rng, residual=r, y=r)
        assert torch.equal(r, y)
    dy = _rand(g, (T, H), 1.0, dtype)
    d_rows = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    dg = torch.empty(T, k, device="cuda")
    B.moe_combine_backward(dy, rows, S, G, p=p, rng=rng, d_out_rows=d_rows, d_gates=dg)
    wr, er, wg, eg = R.combine_backward(R.f64(dy), R.f64(rows), slot_row, gd, m, dtype)
    named = ~np.isnan(wr[:, 0])
    _near(d_rows[torch.from_numpy(named).cuda()], wr[named], er[named], "d_rows")
    assert (d_rows[torch.from_numpy(~named).cuda()] == 7).all()
    _near(dg, wg, eg, "d_gates")
    dg2, dr2 = torch.empty_like(dg), torch.full_like(d_rows, 7.0)
    B.moe_combine_backward(dy, rows, S, G, p=p, rng=rng, d_gates=dg2)
    B.moe_combine_backward(dy, rows, S, G, p=p, rng=rng, d_out_rows=dr2)
    assert torch.equal(dg, dg2) and torch.equal(d_rows, dr2)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_combine_dropped_places_hide_nan(B, dtype):
    """A dropped element is 0 (plus the residual) whatever the rows or dy hold."""
    T, H, k, p = 12, 64, 2, 0.5
    g, rows, slot_row, gates = _combine_inputs(T, H, k, dtype, 2)
    rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    S, G = torch.from_numpy(slot_row).cuda(), torch.from_numpy(gates).cuda()
    rows.fill_(float("nan"))
    y = B.moe_combine_dropout(rows, S, G, p=p, rng=rng)
    m = torch.from_numpy(R.keep(5, 6, T, H, p)).cuda()
    live = torch.from_numpy((slot_row >= 0).any(1)).cuda()
    assert (y[~m] == 0).all() and y[m & live[:, None]].isnan().all()
    dy = torch.where(m, 1.0, float("nan")).to(dtype)
    dr = torch.zeros(T * k, H, dtype=dtype, device="cuda")
    B.moe_combine_backward(dy, torch.ones_like(rows), S, G, p=p, rng=rng, d_out_rows=dr,
                           d_gates=(dg := torch.empty(T, k, device="cuda")))
    assert not dr.isnan().any() and not dg.isnan().any()


def test_combine_without_dropout_is_moe_combine(B):
    for dtype in (BF16, F32):
        g, rows, slot_row, gates = _combine_inputs(50, 256, 8, dtype, 3)
        S, G = torch.from_numpy(slot_row).cuda(), torch.from_numpy(gates).cuda()
        assert torch.equal(B.moe_combine_dropout(rows, S, G), B.moe_combine(rows, S, G))


# --------------------------------------------------- offsets beyond 32 bits
FAR = 64  # rows looked at, at either end of the long arrays


def _ends(T):
    return torch.cat([torch.arange(FAR), torch.arange(T - FAR, T)]).cuda()


def test_linear_with_more_than_2_31_elements(B):
    """Rows beyond 2^31 elements of y, z, dy and dz; dy is 0 but for the rows at
    the ends, so that dw and dbias are those rows' sums."""
    T, K, O, act = 1 << 20, 64, 2056, "silu"
    at = _ends(T)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, generator=gen, device="cuda").to(BF16)
    w = (torch.randn(O, K, generator=gen, device="cuda") / 8).to(BF16)
    ws = B.new_workspace(max(B.moe_linear_workspace_size(T, K, O, act, BF16),
                             B.moe_linear_backward_workspace_size(T, K, O, act, BF16)), "cuda")
    z = torch.empty(T, O, dtype=BF16, device="cuda")
    y = B.moe_linear(x, w, ws, act=act, z=z)
    yr, zr, ey, ez = R.linear(R.f64(x[at]), R.f64(w), None, None, act, BF16)
    _near(z[at], zr, ez, "z")
    _near(y[at], yr, ey, "y")
    dy = y.zero_()
    dy[at] = torch.randn(2 * FAR, O, generator=gen, device="cuda").to(BF16)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(O, dtype=BF16, device="cuda")
    B.moe_linear_backward(dy, x, w, ws, z=z, act=act, dx=dx, dw=dw, dbias=db)
    r = R.linear_backward(R.f64(dy[at]), R.f64(x[at]), R.f64(w), R.f64(z[at]), act, BF16)
    _near(dx[at], *r["dx"], "dx")
    _near(dw, *r["dw"], "dw")  # the zeros between the ends add no rounding
    _near(db, *r["db"], "db")
    dx[at] = 0
    assert not dx.any()


def test_combine_with_more_than_2_31_elements(B):
    T, k, H, p = 140000, 8, 2048, 0.25
    at = _ends(T)
    gen = torch.Generator(device="cuda").manual_seed(4)
    S = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).view(T, k)  # the last rows first
    G = torch.rand(T, k, generator=gen, device="cuda")
    rows = torch.zeros(T * k, H, dtype=BF16, device="cuda")
    named = S[at].long().reshape(-1)
    rows[named] = torch.randn(len(named), H, generator=gen, device="cuda").to(BF16)
    dy = torch.randn(T, H, generator=gen, device="cuda").to(BF16)
    rng = torch.tensor([8, 9], dtype=torch.int64, device="cuda")
    y = B.moe_combine_dropout(rows, S, G, p, rng)
    d_rows, dg = torch.empty_like(rows), torch.empty_like(G)
    B.moe_combine_backward(dy, rows, S, G, p, rng, d_out_rows=d_rows, d_gates=dg)
    blocks = H // 4
    keep = np.stack([[wd >= int(p * 2 ** 32) for b in range(t * blocks, (t + 1) * blocks) for wd in R.philox(8, 9, b)]
                     for t in at.tolist()])
    m = keep / (1 - p)
    local = np.arange(2 * FAR * k, dtype=np.int32).reshape(2 * FAR, k)
    sub, gd = R.f64(rows[named]), R.f64(G[at])
    want, e = R.combine(sub, local, gd, None, m, BF16)
    _near(y[at], want, e, "y")
    wr, er, wg, eg = R.combine_backward(R.f64(dy[at]), sub, local, gd, m, BF16)
    _near(d_rows[named], wr, er, "d_rows")
    _near(dg[at], wg, eg, "d_gates")


def test_router_losses_of_the_largest_batch(B):
    """2^20 tokens of 1024 experts (2^32 bytes of scores): the gates' gradient of
    the tokens at the ends, counts and means of all of them."""
    T, N, k = 1 << 20, 1024, 2
    at = _ends(T)
    gen = torch.Generator(device="cuda").manual_seed(5)
    L = torch.randn(T, N, generator=gen, device="cuda")
    S = torch.randint(0, N, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    DG = torch.randn(T, k, generator=gen, device="cuda")
    out = B.moe_balance_loss(L, S, B.new_workspace(B.moe_balance_workspace_size(T, N), "cuda"))
    assert torch.equal(out["counts"][:N].long(), torch.bincount(S.reshape(-1), minlength=N))
    assert int(out["counts"][N]) == T
    lse = torch.logsumexp(L.double(), 1)
    e = (R.ACT + N / 16 + 12) * R.U  # |z| < 6: the bound of the small batches
    assert float((out["lse"].double() - lse).abs().max()) <= e + R.U * float(lse.max())
    mean = torch.zeros(N, dtype=torch.float64, device="cuda")
    for i in range(0, T, 1 << 17):
        mean += torch.exp(L[i:i + (1 << 17)].double() - lse[i:i + (1 << 17), None]).sum(0)
    mean /= T
    assert float(((out["mean_prob"].double() - mean).abs() / mean).max()) <= 2 * e
    dz = B.moe_router_backward(L, S, out["lse"], out["counts"], d_gates=DG)
    r = R.balance(R.f64(L[at]), S[at].cpu().numpy(), None, None, R.f64(DG[at]))
    _near(dz[at], r["dlogits"], 6 * e * r["scale"] + R.U * np.abs(r["dlogits"]) * 1.01, "dlogits")


# ------------------------------------------------- together, streams, graphs
class _Step:
    """One tuning step of a router and a shared expert beside frozen routed
    experts, as a user's program runs it: forward, losses, and the gradients of
    the router's and the shared expert's weights."""

    def __init__(self, B, T=96, H=256, N=16, k=4, I=128, dtype=BF16, seed=0):
        self.B, self.k, self.N, self.T = B, k, N, T
        g = np.random.default_rng(seed)
        c = lambda *s: _rand(g, s, s[-1] ** -0.5, dtype)  # noqa: E731
        self.x, self.target = _rand(g, (T, H), 1.0, dtype), _rand(g, (T, H), 1.0, dtype)
        self.wg, self.w13, self.w2 = c(N, H), c(N, 2 * I, H), c(N, H, I)
        self.s13, self.s2, self.b2 = c(2 * I, H), c(H, I), _rand(g, (H,), 0.1, dtype)
        self.mask = torch.ones(T, dtype=torch.uint8, device="cuda")
        self.mask[-5:] = 0
        self.rng = torch.tensor([11, 0], dtype=torch.int64, device="cuda")
        self.d_losses = torch.tensor([0.02, 0.001], device="cuda")
        self.p = 0.1
        e = lambda *s: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        n = lambda size: B.new_workspace(size, "cuda")  # noqa: E731
        lay = B.Layer(T, H, N, k, I, 0, dtype)
        self.lay = lay
        self.ws_router = n(B.moe_router_workspace_size(T, N, H, dtype))
        self.ws = n(max(B.moe_linear_workspace_size(T, H, I, "swiglu", dtype),
                        B.moe_linear_workspace_size(T, I, H, "none", dtype),
                        B.moe_linear_backward_workspace_size(T, H, I, "swiglu", dtype),
                        B.moe_linear_backward_workspace_size(T, I, H, "none", dtype),
                        B.moe_linear_backward_workspace_size(T, H, N, "none", dtype),
                        B.moe_balance_workspace_size(T, N), B.moe_ffn_workspace_size(T, N, k, H, I, dtype)))
        self.z, self.h, self.shared, self.y = e(T, 2 * I), e(T, I), e(T, H), e(T, H)
        self.logits = torch.empty(T, N, device="cuda")
        self.loss = dict(losses=torch.empty(2, device="cuda"),
                         counts=torch.empty(N + 1, dtype=torch.int32, device="cuda"),
                         mean_prob=torch.empty(N, device="cuda"), lse=torch.empty(T, device="cuda"))
        self.dy, self.dg, self.dl = e(T, H), torch.empty(T, k, device="cuda"), e(T, N)
        self.dh = e(T, I)
        self.grads = dict(wg=e(N, H), s13=e(2 * I, H), s2=e(H, I), b2=e(H), xr=e(T, H), xs=e(T, H))

    def run(self):
        B, lay, k = self.B, self.lay, self.k
        B.moe_router_topk(self.x, self.wg, k, 0, self.ws_router, self.logits, lay.topk_ids,
                          lay.topk_gates, lay.fallback_ids)
        B.moe_dispatch(lay.topk_ids, self.N, lay.ws_disp, lay.disp)
        B.moe_expert_ffn(self.x, lay.disp["row_token"], lay.disp["expert_offsets"], self.w13, self.w2,
                         k, self.ws, lay.out_rows)
        B.moe_linear(self.x, self.s13, self.ws, act="swiglu", z=self.z, y=self.h)
        B.moe_linear(self.h, self.s2, self.ws, bias=self.b2, residual=self.x, y=self.shared)
        B.moe_combine_dropout(lay.out_rows, lay.disp["slot_row"], lay.topk_gates, self.p, self.rng,
                              self.shared, self.y)
        B.moe_balance_loss(self.logits, lay.topk_ids, self.ws, self.mask, self.loss)
        torch.sub(self.y, self.target, out=self.dy)
        self.dy.mul_(self.mask[:, None])
        B.moe_combine_backward(self.dy, lay.out_rows, lay.disp["slot_row"], lay.topk_gates, self.p,
                               self.rng, d_gates=self.dg)
        B.moe_router_backward(self.logits, lay.topk_ids, self.loss["lse"], self.loss["counts"],
                              self.d_losses, self.mask, self.dg, self.dl)
        G = self.grads
        B.moe_linear_backward(self.dl, self.x, self.wg, self.ws, dx=G["xr"], dw=G["wg"])
        B.moe_linear_backward(self.dy, self.h, self.s2, self.ws, dx=self.dh, dw=G["s2"], dbias=G["b2"])
        B.moe_linear_backward(self.dh, self.x, self.s13, self.ws, z=self.z, act="swiglu", dx=G["xs"],
                              dw=G["s13"])

    def outputs(self):
        return {"y": self.y, "losses": self.loss["losses"], "counts": self.loss["counts"], **self.grads}


def test_tuning_step_against_autograd(B):
    """The step's gradients against a 64-bit autograd of the same step (same
    routing, mask and expert rows).  Every intermediate that the kernels hand on
    in bf16 (h, z, the shared output, y, dy, dlogits, dh) is off by half a step,
    2^-8; a dozen such roundings along a chain keep the relative error of a whole
    gradient tensor (2-norm) under 12 2^-8."""
    st = _Step(B)
    st.run()
    T, k = st.T, st.k
    lay = st.lay
    D = lambda t: t.detach().double().cpu()  # noqa: E731
    x0, wg, s13, s2, b2 = (D(t).requires_grad_() for t in (st.x, st.wg, st.s13, st.s2, st.b2))
    xr = D(st.x).requires_grad_()
    ids, slot_row = lay.topk_ids.cpu().long(), lay.disp["slot_row"].cpu().long()
    logits = xr @ wg.t()
    prob = torch.softmax(logits, 1)
    gates = prob.gather(1, ids)
    rows = D(lay.out_rows)[slot_row]
    z = x0 @ s13.t()
    I = z.shape[1] // 2
    hh = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
    shared = hh @ s2.t() + b2 + D(st.x)
    m = torch.from_numpy(R.keep(11, 0, T, x0.shape[1], st.p) / (1 - st.p))
    y = shared + m * (gates[:, :, None] * rows).sum(1)
    on = st.mask.cpu().double()
    n = on.sum()
    counts = torch.zeros(st.N, dtype=torch.float64)
    for t in range(T):
        if on[t]:
            counts[ids[t]] += 1
    bal = st.N / (k * n) * (counts * (prob * on[:, None]).sum(0) / n).sum()
    zl = ((torch.logsumexp(logits, 1) ** 2) * on).sum() / n
    total = 0.5 * (((y - D(st.target)) ** 2) * on[:, None]).sum() + 0.02 * bal + 0.001 * zl
    total.backward()
    assert np.array_equal(st.loss["counts"].cpu().numpy()[:-1], counts.numpy().astype(np.int64))
    want = dict(wg=wg.grad, s13=s13.grad, s2=s2.grad, b2=b2.grad, xr=xr.grad, xs=x0.grad, y=y.detach())
    for name, v in want.items():
        got = D(st.outputs()[name])
        rel = float((got - v).norm() / v.norm())
        print(f"[gpu-test] step {name}: {rel:.2e}", flush=True)
        assert rel <= 12 * 2.0 ** -8, (name, rel)


def test_tuning_step_on_a_side_stream(B):
    st = _Step(B, seed=1)
    st.run()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in st.outputs().items()}
    for t in st.outputs().values():
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        st.run()
    side.synchronize()
    for n, t in st.outputs().items():
        assert torch.equal(t, want[n]), n


def test_tuning_steps_captured_with_one_workspace(B):
    """Two captured steps that share a workspace, replayed in turn with eager
    work between; the dropout offset and the inputs change between replays, and
    every replay equals the eager step."""
    a, b = _Step(B, seed=2), _Step(B, T=80, seed=3)
    if b.ws.numel() > a.ws.numel():
        a.ws = b.ws
    b.ws = a.ws
    graphs = []
    for st in (a, b):
        st.run()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            st.run()
        graphs.append(gr)
    seen = []
    for rep in range(4):
        for st, gr in zip((a, b), graphs):
            st.rng[1] = 100 + rep
            st.x.mul_(-1 if rep % 2 else 1.0)
            st.run()
            torch.cuda.synchronize()
            want = {n: t.clone() for n, t in st.outputs().items()}
            for t in st.outputs().values():
                t.zero_()
            gr.replay()
            torch.cuda.synchronize()
            for n, t in st.outputs().items():
                assert torch.equal(t, want[n]), (rep, n)
            if st is a:
                seen.append(want["y"])
    assert not torch.equal(seen[0], seen[2])  # another offset, another mask


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_gradients_without_the_inputs_they_do_not_need(B, dtype):
    """dx without x, dw and dbias without w, d_out_rows without out_rows, the
    losses' gradient without topk_ids: the same bits as with them."""
    T, K, O = 70, 72, 136
    g, x, w, _, _ = _linear_inputs(T, K, O, "silu", dtype, 21, False, False)
    dy, z = _rand(g, (T, O), 0.5, dtype), _rand(g, (T, O), 1.0, dtype)
    ws = B.new_workspace(B.moe_linear_backward_workspace_size(T, K, O, "silu", dtype), "cuda")
    e = torch.empty_like
    for names, xa, wa in ((("dx",), None, w), (("dw", "dbias"), x, None), (("dbias",), None, w)):
        full = {n: {"dx": e(x), "dw": e(w), "dbias": e(w[:, 0])}[n] for n in names}
        part = {n: e(t) for n, t in full.items()}
        B.moe_linear_backward(dy, x, w, ws, z=z, act="silu", **full)
        B.moe_linear_backward(dy, xa, wa, ws, z=z, act="silu", **part)
        assert all(torch.equal(full[n], part[n]) for n in names)
    g, rows, slot_row, gates = _combine_inputs(9, 64, 3, dtype, 4)
    S, G, dyc = torch.from_numpy(slot_row).cuda(), torch.from_numpy(gates).cuda(), _rand(g, (9, 64), 1.0, dtype)
    a, b = torch.zeros_like(rows), torch.zeros_like(rows)
    B.moe_combine_backward(dyc, rows, S, G, d_out_rows=a)
    B.moe_combine_backward(dyc, None, S, G, d_out_rows=b)
    assert torch.equal(a, b)
    _, logits, ids = _balance_inputs(33, 20, 3, 6)
    L, ids = torch.from_numpy(logits).cuda(), torch.from_numpy(ids).cuda()
    out = B.moe_balance_loss(L, ids, B.new_workspace(B.moe_balance_workspace_size(33, 20), "cuda"))
    dl = torch.tensor([0.5, 0.25], device="cuda")
    assert torch.equal(B.moe_router_backward(L, ids, out["lse"], out["counts"], dl, dtype=dtype),
                       B.moe_router_backward(L, None, out["lse"], out["counts"], dl, dtype=dtype, k=3))


def test_binding_refusals_on_the_gpu(B):
    x, w = torch.zeros(4, 64, device="cuda"), torch.zeros(32, 64, device="cuda")
    ws = B.new_workspace(1 << 16, "cuda")
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_linear(x.t().contiguous().t(), w, ws)
    with pytest.raises(ValueError, match="shape"):
        B.moe_linear(x, w, ws, bias=torch.zeros(31, device="cuda"))
    with pytest.raises(ValueError, match="dtype"):
        B.moe_linear(x, w.bfloat16(), ws)
    with pytest.raises(RuntimeError, match="EUNSUP"):
        B.moe_linear(torch.zeros(4, 62, device="cuda"), torch.zeros(32, 62, device="cuda"), ws)
    flat = torch.zeros(4 * 64 + 1, device="cuda")
    with pytest.raises(RuntimeError, match="EINVAL"):
        B.moe_linear(flat[1:].view(4, 64), w, ws)
    with pytest.raises(RuntimeError, match="EINVAL"):
        B.moe_linear_backward(torch.zeros(4, 32, device="cuda"), x, w, ws[:16], dw=w.clone(),
                              dbias=torch.zeros(32, device="cuda"))
    rows, S, G = torch.zeros(8, 64, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), \
        torch.zeros(4, 2, device="cuda")
    with pytest.raises(RuntimeError, match="EINVAL"):
        B.moe_combine_dropout(rows, S, G, p=1.0, rng=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="dropout needs rng"):
        B.moe_combine_dropout(rows, S, G, p=0.5)
