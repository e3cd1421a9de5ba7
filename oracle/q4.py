"""The 4-bit decode operators and the log probabilities in 64 bits (numpy),
from the formulas and byte layouts that include/tqd.h states.  The oracle of
the operator tests; the library never uses it."""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ formats

def quantise_groups(y):
    """y [..., 32 * m] -> codes uint8 (1..15), scales f16 [..., m]; groups that
    hold a NaN or an infinity, or whose scale passes f16, get a NaN scale."""
    y = np.asarray(y, dtype=np.float64)
    g = y.reshape(*y.shape[:-1], -1, 32)
    a = np.abs(g).max(-1)
    with np.errstate(all="ignore"):
        d = np.float32(a / 7)
        bad = ~(d < 65520)
        q = np.rint(7 * g / np.where(a > 0, a, 1)[..., None])
        q = np.where(bad[..., None], 0, q)
        scales = np.where(bad, np.float16(np.nan), d.astype(np.float16))
    return (q + 8).astype(np.uint8).reshape(y.shape), scales


def group_values(codes, scales):
    g = (codes.astype(np.float64) - 8).reshape(*codes.shape[:-1], -1, 32)
    return (g * scales.astype(np.float64)[..., None]).reshape(codes.shape)


def rotate(x, pos, table):
    """Half-split rotation of x [n, heads, hd] at positions pos [n], table f32 [max_pos, hd / 2, 2]."""
    x = np.asarray(x, dtype=np.float64)
    half = x.shape[-1] // 2
    c = table[pos, :, 0].astype(np.float64)[:, None]
    s = table[pos, :, 1].astype(np.float64)[:, None]
    return np.concatenate([x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s], -1)


def page_bytes(n_kv, hd, page_size):
    return n_kv * page_size * hd * 9 // 8


def _nibble_places(b, hd):
    """For block position b: (byte, shift) of every element's K code and V code,
    and the bytes of the K and V scales."""
    ng, d = hd // 32, np.arange(hd)
    g, c, i = d // 32, d % 32 // 8, d % 8
    row = 8 * ((b // 2) % 2) + 2 * (b // 4) + b % 2
    k = row * (hd // 2) + 4 * (c * ng + g) + i // 2, 4 * (i % 2)
    n, nib = d % 8, d // 8
    if hd == 128:
        piece = 512 * ((b // 2) % 2) + 128 * (b // 4) + 16 * n + 8 * (b % 2)
    else:
        piece = 128 * (b // 4) + 16 * n + 4 * (b % 4)
    v = 9 * hd + piece + nib // 2, 4 * (nib % 2)
    ks = 8 * hd + 2 * (b * ng + np.arange(ng))
    vs = 17 * hd + 2 * (b * ng + np.arange(ng))
    return k, v, ks, vs


def _block(pages, page, h, pos_in_page, page_size, hd):
    per_head = page_size * hd * 9 // 8
    at = h * per_head + pos_in_page // 16 * 18 * hd
    return pages[page, at:at + 18 * hd]


def store_row(pages, page, h, pos_in_page, page_size, kc, ks, vc, vs):
    """Write one position's codes [hd] and scales [hd / 32] of one head into pages uint8 [n_pages, page bytes]."""
    hd = kc.size
    blk = _block(pages, page, h, pos_in_page, page_size, hd)
    (kb, ksh), (vb, vsh), ksb, vsb = _nibble_places(pos_in_page % 16, hd)
    for at, sh, code in ((kb, ksh, kc), (vb, vsh, vc)):
        blk[at] = 0
        np.bitwise_or.at(blk, at, (code << sh).astype(np.uint8))
    for at, s in ((ksb, ks), (vsb, vs)):
        raw = np.ascontiguousarray(s, dtype=np.float16).view(np.uint8).reshape(-1, 2)
        blk[at], blk[at + 1] = raw[:, 0], raw[:, 1]


def load_row(pages, page, h, pos_in_page, page_size, hd):
    """(K values, V values, K scales, V scales) of one position of one head."""
    blk = _block(pages, page, h, pos_in_page, page_size, hd)
    (kb, ksh), (vb, vsh), ksb, vsb = _nibble_places(pos_in_page % 16, hd)
    f16 = lambda at: np.stack([blk[at], blk[at + 1]], -1).reshape(-1).view(np.float16)  # noqa: E731
    ks, vs = f16(ksb), f16(vsb)
    return (group_values((blk[kb] >> ksh) & 15, ks), group_values((blk[vb] >> vsh) & 15, vs), ks, vs)


def q4_0_blocks(codes, d):
    """codes uint8 [rows, cols] (0..15), d f16 [rows, cols / 32] -> 18-byte blocks [rows, cols / 32 * 18]."""
    rows, cols = codes.shape
    c = codes.reshape(rows, cols // 32, 2, 16)
    raw = np.ascontiguousarray(d, dtype=np.float16).view(np.uint8).reshape(rows, cols // 32, 2)
    return np.concatenate([raw, c[:, :, 0] | (c[:, :, 1] << 4)], -1).reshape(rows, -1)


def q4_0_values(codes, d):
    return group_values(codes, d)


def q4_0_tiles(codes, d):
    """The library's tile layout, element by element from its description."""
    rows, cols = codes.shape
    rt, st = -(-rows // 16), -(-cols // 128)
    words = np.full((rt, st, 16, 4, 4), 0x88888888, dtype=np.uint32)
    scales = np.zeros((rt, st, 16, 4), dtype=np.float16)
    for r in range(rows):
        for g in range(cols // 32):
            scales[r // 16, g // 4, r % 16, g % 4] = d[r, g]
            for c in range(4):
                w = 0
                for i in range(8):
                    w |= int(codes[r, 32 * g + 8 * c + i]) << (4 * i)
                words[r // 16, g // 4, r % 16, c, g % 4] = w
    raw = np.concatenate([words.reshape(rt, st, -1).view(np.uint8).reshape(rt, st, -1),
                          scales.reshape(rt, st, -1).view(np.uint8).reshape(rt, st, -1)], -1)
    return raw.reshape(-1)


# ------------------------------------------------------------------ operators

def attention(q, K, V, visible):
    """q [heads, hd], K, V [T, n_kv, hd], the first `visible` positions seen: [heads, hd]."""
    heads, hd = q.shape
    n_kv = K.shape[1]
    out = np.zeros((heads, hd))
    if visible <= 0:
        return out
    for h in range(heads):
        k, v = K[:visible, h // (heads // n_kv)], V[:visible, h // (heads // n_kv)]
        s = k @ q[h] / np.sqrt(hd)
        p = np.exp(s - s.max())
        out[h] = p @ v / p.sum()
    return out


def logprobs(x, target, top_k):
    """(log p of target, entropy, ids, their log p) of one row; also E[|d|], E[d^2] of d = x - max for the error bound."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64))
    m = x.max()
    ids = np.full(top_k, -1)
    tops = np.full(top_k, -np.inf)
    if m == -np.inf:
        return -np.inf, 0.0, ids, tops, 0.0, 0.0
    with np.errstate(invalid="ignore"):
        d = np.where(x == m, 0.0, x - m)
    e = np.exp(d)
    s = e.sum()
    lp = d - np.log(s)
    p = e / s
    dz = np.where(p > 0, d, 0.0)
    order = np.argsort(-x, kind="stable")[:top_k]
    order = order[x[order] > -np.inf]
    ids[:order.size] = order
    tops[:order.size] = lp[order]
    at = lp[target] if 0 <= target < x.size else np.nan
    return at, float(np.log(s) - (p * dz).sum()), ids, tops, float((p * np.abs(dz)).sum()), float((p * dz * dz).sum())
