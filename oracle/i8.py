"""Rows of 8-bit codes, their products, and rotations of many rows, in 64 bits
(numpy), from the formulas that include/tqd.h states.  The oracle of the
operator tests; the library never uses it."""
from __future__ import annotations

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def rows(y, factor=1.0):
    """y [n, w] (f64) -> codes int8 and scales (f64, not yet rounded) of factor [n, 1] * y; the codes go by y alone."""
    y = np.asarray(y, dtype=np.float64)
    with np.errstate(all="ignore"):
        most = np.abs(y).max(1, keepdims=True)
        bad = ~(np.isfinite(y).all(1, keepdims=True)) | ~(np.abs(np.float32(most * factor)) <= F32_MAX)
        t = 127 * y / np.where(most > 0, most, 1)
        q = np.rint(t)
        low = np.floor(t)
        # next to a border the quotient's own rounding may decide: there by products, of 56 bits at most where y has 48
        at = np.nonzero(np.abs(t - low - 0.5) < 1e-9)
        row_most = np.broadcast_to(most, y.shape)[at].astype(np.longdouble)
        side = 127 * y[at].astype(np.longdouble) - (low[at] + 0.5) * row_most
        q[at] = np.where(side == 0, low[at] + (low[at] % 2), low[at] + (side > 0))
        q = np.where(bad, 0, q).astype(np.int8)
        scale = np.where(bad, np.nan, most * factor / 127)
    return q, scale[:, 0]


def norm_rows(x, add, g, eps):
    """Sum f32, codes and scales of the RMSNorm of x + add (f32 arrays)."""
    with np.errstate(all="ignore"):
        h = (x if add is None else x + add).astype(np.float32)
        d = h.astype(np.float64)
        at = (d * d).mean(1, keepdims=True) + np.float64(np.float32(eps))
        q, s = rows(d * g.astype(np.float64), np.where(at > 0, 1 / np.sqrt(np.where(at > 0, at, 1)), 0))
    return h, q, s


def silu_rows(gate, up):
    with np.errstate(all="ignore"):
        g = gate.astype(np.float64)
        return rows(g / (1 + np.exp(-g)) * up.astype(np.float64))


def matmul(w, w_scale, x, x_scale):
    """The exact sums (of whole numbers below 2^53, so exact in f64), and the f32 result of their stated roundings."""
    s = x.astype(np.float64) @ w.astype(np.float64).T
    with np.errstate(all="ignore"):
        return s, s.astype(np.float32) * x_scale.astype(np.float32)[:, None] * w_scale.astype(np.float32)[None]


def rope_table(theta, d, n, kind=0, factor=1.0, original=0, low=1.0, high=32.0, attention=1.0):
    """[n, d / 2, 2] in f64.  The arguments as the library takes them: f32 numbers."""
    theta, factor, low, high, attention = (float(np.float32(v)) for v in (theta, factor, low, high, attention))
    i = np.arange(d // 2)
    f = theta ** (-2.0 * i / d)
    keep = np.ones(d // 2)
    if kind == 1:
        keep[:] = 0
    if kind == 2:
        keep = (original * f / (2 * np.pi) - low) / (high - low)
    if kind == 3:
        index = lambda r: d / 2 * np.log(original / (2 * np.pi * r)) / np.log(theta)  # noqa: E731
        a, b = max(np.floor(index(high)), 0), min(np.ceil(index(low)), d - 1)
        keep = 1 - (i - a) / (b - a if b > a else 0.001)
    keep = np.clip(keep, 0, 1)
    angle = np.arange(n)[:, None] * (f * (keep + (1 - keep) / (factor if kind else 1)))[None]
    return attention * np.stack([np.cos(angle), np.sin(angle)], -1)


def rope_rows(x, heads, pos, table, interleaved):
    """x [n, heads * hd] turned by table [.., d / 2, 2] at pos [n] (all f64), and the size of each sum's terms."""
    n, half = x.shape[0], table.shape[1]
    x = np.asarray(x, dtype=np.float64).reshape(n, heads, -1)
    out, size = x.copy(), np.zeros_like(x)
    a = np.arange(half)
    p, q = (2 * a, 2 * a + 1) if interleaved else (a, a + half)
    c, s = table[pos][:, None, :, 0], table[pos][:, None, :, 1]
    out[..., p] = x[..., p] * c - x[..., q] * s
    out[..., q] = x[..., q] * c + x[..., p] * s
    size[..., p] = np.abs(x[..., p] * c) + np.abs(x[..., q] * s)
    size[..., q] = np.abs(x[..., q] * c) + np.abs(x[..., p] * s)
    return out.reshape(n, -1), size.reshape(n, -1)
