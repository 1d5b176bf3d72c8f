"""Plain 64-bit definitions of the dense layer, the router's losses and the
training combine, with the rounding bounds that the GPU results are held to.

A bound is the sum of
  - half a step of the output type relative to the value (bf16 2^-8, fp32 2^-24);
  - for a sum of n products in fp32, n 2^-24 times the sum of their absolute values;
  - for an activation in fp32, a few units: ACT 2^-24 times (|z| + 1) (the
    exponential's argument is rounded, which costs |z| 2^-24 relative);
  - where an operand of a product is rounded to the element type first (dz),
    half a step of each operand times the sum of the absolute products.
"""
from __future__ import annotations

import numpy as np
import torch
from scipy.special import erf, expit

U = 2.0 ** -24
ACT = 24


def half(dtype) -> float:
    """Half a step relative to the value."""
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def f64(t) -> np.ndarray | None:
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def product(a, b):
    """a @ b in 64 bits, on the GPU where it is large."""
    if a.shape[0] * a.shape[1] * b.shape[1] > 1 << 31 and torch.cuda.is_available():
        return (torch.from_numpy(np.ascontiguousarray(a)).cuda()
                @ torch.from_numpy(np.ascontiguousarray(b)).cuda()).cpu().numpy()
    return a @ b


# --------------------------------------------------------------------- linear
def act_value(z, act):
    if act == "relu":
        return np.maximum(z, 0)
    if act == "silu":
        return z * expit(z)
    if act == "gelu":
        return z * 0.5 * (1 + erf(z / np.sqrt(2)))
    return z


def act_slope(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        s = expit(z)
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + erf(z / np.sqrt(2))) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    return np.ones_like(z)


def linear(x, w, bias, residual, act, dtype):
    """(y, z, bound of y, bound of z); arguments fp64."""
    K = x.shape[1]
    b = 0.0 if bias is None else bias
    z = product(x, w.T) + b
    ez = (K + 2) * U * (product(np.abs(x), np.abs(w).T) + np.abs(b))
    if act == "swiglu":
        O = w.shape[0] // 2
        g, u = z[:, :O], z[:, O:]
        eg, eu = ez[:, :O], ez[:, O:]
        y = act_value(g, "silu") * u
        # |silu'| <= 1.1; the products of the errors are covered by the activation's units
        ey = 1.1 * eg * np.abs(u) + np.abs(act_value(g, "silu")) * eu + 1.1 * eg * eu
        ey += ACT * U * (np.abs(g) + 1) * (np.abs(u) + eu)
    else:
        y = act_value(z, act)
        # |gelu'| <= 1.13
        ey = 1.13 * ez + (0 if act in ("none", "relu") else ACT * U * (np.abs(z) + 1))
    if residual is not None:
        y = y + residual
        ey = ey + U * np.abs(y)
    h = half(dtype)
    return y, z, ey * (1 + h) + h * np.abs(y), ez * (1 + h) + h * np.abs(z)


def act_grad(dy, z, act):
    """(dz, its fp32 bound)."""
    if act == "none":
        return dy, np.zeros_like(dy)
    if act == "swiglu":
        O = dy.shape[1]
        g, u = z[:, :O], z[:, O:]
        dz = np.concatenate([dy * u * act_slope(g, "silu"), dy * act_value(g, "silu")], 1)
        e = ACT * U * (np.abs(g) + 1) * np.abs(dy)
        return dz, np.concatenate([e * (np.abs(u) * (np.abs(g) + 1)), e], 1)
    dz = dy * act_slope(z, act)
    return dz, ACT * U * (np.abs(z) + 1) ** 2 * np.abs(dy)


def linear_backward(dy, x, w, z, act, dtype):
    """dict of (value, bound) of dx, dw, db."""
    dz, e = act_grad(dy, z, act)
    h = half(dtype)
    ez = e + (0 if act == "none" else h * (np.abs(dz) + e))
    T, W = dz.shape
    out = {}
    for name, a, ea, b, n in (("dx", dz, ez, w, W), ("dw", dz.T, ez.T, x, T)):
        v = product(a, b)
        err = product(ea + (n + 2) * U * (np.abs(a) + ea), np.abs(b))
        out[name] = (v, err * (1 + h) + h * np.abs(v))
    v = dz.sum(0)
    err = e.sum(0) + (T + 2) * U * (np.abs(dz) + e).sum(0)
    out["db"] = (v, err * (1 + h) + h * np.abs(v))
    return out


# -------------------------------------------------------------------- balance
def balance(logits, ids, mask, d_losses=None, d_gates=None):
    """The losses, statistics and the logits' gradient, token by token."""
    T, N = logits.shape
    k = ids.shape[1]
    on = np.ones(T, bool) if mask is None else mask != 0
    n = int(on.sum())
    counts = np.zeros(N + 1, np.int64)
    counts[N] = n
    prob = np.zeros((T, N))
    lse = np.zeros(T)
    for t in range(T):
        if not on[t]:
            continue
        for j in ids[t]:
            if 0 <= j < N:
                counts[j] += 1
        top = logits[t].max()
        if top == -np.inf:
            lse[t] = -np.inf
            continue
        e = np.exp(logits[t] - top)
        prob[t] = e / e.sum()
        lse[t] = top + np.log(e.sum())
    some = on & np.isfinite(lse)
    inv = 1.0 / n if n else 0.0
    mean_prob = prob.sum(0) * inv
    losses = np.array([N / k * inv * (counts[:N] * mean_prob).sum(), (lse[some] ** 2).sum() * inv])
    out = dict(losses=losses, counts=counts, mean_prob=mean_prob, lse=lse)
    dl = np.zeros(2) if d_losses is None else d_losses
    dz = np.zeros((T, N))
    scale = np.zeros((T, N))
    for t in np.flatnonzero(some):
        u = dl[0] * N * counts[:N] / k * inv * inv
        if d_gates is not None:
            u = u.copy()
            for s, j in enumerate(ids[t]):
                if 0 <= j < N:
                    u[j] += d_gates[t, s]
        dz[t] = prob[t] * (u - (prob[t] * u).sum()) + dl[1] * 2 * lse[t] * prob[t] * inv
        scale[t] = prob[t] * (np.abs(u) + (prob[t] * np.abs(u)).sum() + np.abs(dl[1] * 2 * lse[t] * inv))
    out["dlogits"], out["scale"] = dz, scale
    return out


# -------------------------------------------------------------------- combine
def philox(seed: int, offset: int, block: int):
    """The four words of one Philox4x32-10 block, in plain integers."""
    m = 0xFFFFFFFF
    c = [block & m, block >> 32, offset & m, (offset >> 32) & m]
    k0, k1 = seed & m, (seed >> 32) & m
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k0, b & m, (a >> 32) ^ c[3] ^ k1, a & m]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return c


def keep(seed, offset, T, H, p):
    thr = int(p * 4294967296.0)
    w = [v for b in range(T * H // 4) for v in philox(seed, offset, b)]
    return np.array(w, dtype=np.uint64).reshape(T, H) >= thr


def combine(rows, slot_row, gates, residual, m, dtype):
    """(y, bound); m: dropout factor per element."""
    T, k = slot_row.shape
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for s in range(k):
            if slot_row[t, s] >= 0:
                y[t] += gates[t, s] * rows[slot_row[t, s]]
                mag[t] += np.abs(gates[t, s] * rows[slot_row[t, s]])
    on = m != 0
    y, mag = np.where(on, y * m, 0), np.where(on, mag * m, 0)
    if residual is not None:
        y, mag = y + residual, mag + np.abs(residual)
    err = (k + 4) * U * mag
    h = half(dtype)
    return y, err * (1 + h) + h * np.abs(y)


def combine_backward(dy, rows, slot_row, gates, m, dtype):
    T, k = slot_row.shape
    H = rows.shape[1]
    d = np.where(m != 0, dy * m, 0)
    d_rows, e_rows = np.full_like(rows, np.nan), np.zeros_like(rows)
    dg, eg = np.zeros((T, k)), np.zeros((T, k))
    h = half(dtype)
    for t in range(T):
        for s in range(k):
            r = slot_row[t, s]
            if r < 0:
                continue
            d_rows[r] = gates[t, s] * d[t]
            e_rows[r] = (h + 4 * U) * np.abs(d_rows[r])
            dg[t, s] = rows[r] @ d[t]
            eg[t, s] = (H + 4) * U * (np.abs(rows[r]) @ np.abs(d[t]))
    return d_rows, e_rows, dg, eg
