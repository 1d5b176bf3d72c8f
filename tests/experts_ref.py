"""Plain 64-bit definitions of the grouped products, the norm and gradient
clipping, with the rounding bounds that the GPU results are held to (the units
of training_ref: U = 2^-24 per fp32 operation, half a step of the output type).

A sum along a row of the norm is a tree: at most 64 values one after another in
a thread, 6 steps in a wave, 16 waves; DEPTH = 100 units of the absolute sum
bound it (fewer for shorter rows: H + 2).
"""
from __future__ import annotations

import numpy as np

import training_ref as R

DEPTH = 100


# -------------------------------------------------------------------- grouped
def rows_of(x, token, lo, hi):
    return x[lo:hi] if token is None else x[token[lo:hi]]


def grouped(x, token, offsets, w, act, dtype):
    """(y, z, bound of y, bound of z) of the rows that the experts have."""
    parts = []
    O = w.shape[1] // 2 if act == "swiglu" else w.shape[1]
    for e in range(len(w)):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            parts.append(R.linear(rows_of(x, token, lo, hi), w[e], None, None, act, dtype))
    if not parts:
        return np.zeros((0, O)), np.zeros((0, w.shape[1])), np.zeros((0, O)), np.zeros((0, w.shape[1]))
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(4))


def grouped_backward(dy, x, token, offsets, w, z, act, dtype):
    """dict of (value, bound) of dx (the experts' rows) and dw."""
    dx, ex = [], []
    dw, ew = np.zeros_like(w), np.zeros_like(w)
    for e in range(len(w)):
        lo, hi = offsets[e], offsets[e + 1]
        if hi == lo:
            continue
        r = R.linear_backward(dy[lo:hi], rows_of(x, token, lo, hi), w[e], z[lo:hi], act, dtype)
        dx.append(r["dx"][0])
        ex.append(r["dx"][1])
        dw[e], ew[e] = r["dw"]
    K = w.shape[2]
    cat = lambda a: np.concatenate(a) if a else np.zeros((0, K))  # noqa: E731
    return dict(dx=(cat(dx), cat(ex)), dw=(dw, ew))


# ----------------------------------------------------------------------- norm
def norm(s, w, b, kind, eps, dtype):
    """dict of (value, bound) of y, mean, rstd for the (already rounded) sum s."""
    H = s.shape[1]
    n = min(H + 2, DEPTH)
    mean = s.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(s), 1))
    em = n * R.U * np.abs(s).mean(1, keepdims=True) if kind == "layer" else np.zeros((len(s), 1))
    c = s - mean
    ec = em + R.U * np.abs(c)
    var = (c * c).mean(1, keepdims=True)
    ev = (2 * np.abs(c) * ec + ec * ec).mean(1, keepdims=True) + (n + 2) * R.U * var + R.U * (var + eps)
    rstd = 1 / np.sqrt(var + eps)
    # the slope of v^-1/2 at the lower end of its interval; 4 units for root and quotient
    low = np.maximum(var + eps - ev, 1e-300)
    er = np.where(var + eps > 2 * ev, 0.5 * ev * low ** -1.5, np.inf) + 4 * R.U * rstd
    h = c * rstd
    eh = ec * (rstd + er) + np.abs(c) * er + 2 * R.U * np.abs(h)
    y = h * w
    ey = eh * np.abs(w) + 2 * R.U * np.abs(y)
    if b is not None:
        y = y + b
        ey = ey + 2 * R.U * (np.abs(y) + np.abs(b))
    hf = R.half(dtype)
    return dict(y=(y, ey * (1 + hf) + hf * np.abs(y)), mean=(mean[:, 0], em[:, 0]), rstd=(rstd[:, 0], er[:, 0]))


def norm_backward(dy, s, w, mean, rstd, dsum, kind, dtype):
    """dict of (value, bound) of dx, dw, db for given statistics."""
    T, H = s.shape
    n = min(H + 2, DEPTH)
    m = mean[:, None] if kind == "layer" else 0.0
    r = rstd[:, None]
    h = (s - m) * r
    eh = 3 * R.U * np.abs(h)
    u = dy * w
    mu = u.mean(1, keepdims=True) if kind == "layer" else np.zeros((T, 1))
    emu = (n + 2) * R.U * np.abs(u).mean(1, keepdims=True)
    muh = (u * h).mean(1, keepdims=True)
    emuh = (n + 6) * R.U * np.abs(u * h).mean(1, keepdims=True)
    dx = r * (u - mu - h * muh)
    ex = r * (emu + np.abs(h) * emuh + eh * (np.abs(muh) + emuh) +
              6 * R.U * (np.abs(u) + np.abs(mu) + np.abs(h * muh)))
    if dsum is not None:
        dx = dx + dsum
        ex = ex + R.U * (np.abs(dx) + np.abs(dsum))
    hf = R.half(dtype)
    out = dict(dx=(dx, ex * (1 + hf) + hf * np.abs(dx)))
    # a thread adds the rows of one of at most 512 workgroups, at most 16 groups join in fp32, the rest in fp64
    chain = -(-T // 512) + 20
    for name, v, e in (("dw", dy * h, np.abs(dy) * eh), ("db", dy, 0.0)):
        q = v.sum(0)
        eq = (e + (chain + 1) * R.U * np.abs(v)).sum(0) + R.U * np.abs(q)
        out[name] = (q, eq * (1 + hf) + hf * np.abs(q))
    return out


# ------------------------------------------------------------------- clipping
def clip(grads, max_norm):
    """(norm, factor) of fp64 arrays."""
    norm = np.sqrt(sum(float((g.astype(np.longdouble) ** 2).sum()) for g in grads))
    return norm, max_norm / norm if norm > max_norm and np.isfinite(norm) else 1.0
