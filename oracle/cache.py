"""Norm, rotation, the 4-bit cache format and decode over it, for the oracle (plain numpy, from
the definitions in include/attn.h).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

Rows are float64 [tokens, heads, d]. The 4-bit format: E2M1 codes, one E4M3 scale per 16
channels, one fp32 scale a tensor; a (page, kv head) block holds its tokens' codes, then their
scales.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_round, e4m3_values

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_E4M3 = e4m3_values()


def norm(x, weight, eps):
    """x / sqrt(mean x^2 + eps) * weight over the last axis, in float64."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def pairs(rot, interleaved):
    """Channel indices (first, second) of the rotated pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, cos_sin, pos, rot, interleaved, dtype=np.float64):
    """Turns the pairs of x [tokens, heads, d] by the angles of pos [tokens]. dtype float32
    rounds every product and sum to fp32, as the 4-bit cache is defined."""
    y = np.array(x, dtype=dtype)
    if rot:
        a, b = pairs(rot, interleaved)
        row = np.asarray(cos_sin)[pos].astype(dtype)[:, None, :]
        c, s = row[..., :rot // 2], row[..., rot // 2:]
        p, q = y[..., a].copy(), y[..., b].copy()
        y[..., a] = p * c - q * s
        y[..., b] = q * c + p * s
    return y


def e2m1_round(x):
    """float32 values to E2M1 codes: nearest, ties to the even code, saturating at 6; the sign
    kept."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    a = np.minimum(np.abs(x), 6.0)
    hi = np.minimum(np.searchsorted(E2M1, a, side="left"), 7)
    lo = np.maximum(hi - 1, 0)
    up, down = E2M1[hi] - a, a - E2M1[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def quantize(y, scale):
    """float32 [..., d] to (code bytes [..., d/2], scale bytes [..., d/16]), every step in
    fp32."""
    y = np.asarray(y, dtype=np.float32)
    xs = y * (np.float32(1.0) / np.float32(scale))
    blk = xs.reshape(*xs.shape[:-1], -1, 16)
    sf = e4m3_round(np.abs(blk).max(-1) / np.float32(6.0))
    s = _E4M3[sf].astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.where(s > 0, e2m1_round(np.where(s > 0, blk / s, np.float32(0.0))), 0)
    codes = codes.astype(np.uint8).reshape(y.shape)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), sf


def split_block(pool, page, d):
    """Views (codes [num, Hkv, page, d/2], scales [num, Hkv, page, d/16]) of a 4-bit pool."""
    cut = page * d // 2
    num, hkv, _ = pool.shape
    return (pool[:, :, :cut].reshape(num, hkv, page, d // 2),
            pool[:, :, cut:].reshape(num, hkv, page, d // 16))


def values(codes, scales, scale):
    """Code and scale bytes to float64 values."""
    c = np.stack([codes & 15, codes >> 4], axis=-1)
    c = c.reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    return v * np.repeat(_E4M3[scales], 16, axis=-1) * float(np.float32(scale))


def slots(pos, table_row, page):
    """(physical page, slot) of context positions."""
    pos = np.asarray(pos)
    return np.asarray(table_row)[pos // page], pos % page


def context(pool_values, table_row, length, page):
    """A sequence's rows [Hkv, length, d] from page values [num, Hkv, page, d]."""
    n = -(-length // page)
    rows = pool_values[np.asarray(table_row)[:n]].transpose(1, 0, 2, 3)
    return rows.reshape(rows.shape[0], -1, rows.shape[-1])[:, :length]


def decode(q, k, v, scale):
    """One query row a head: q [Hq, d], k, v [Hkv, n, d] (float64). Returns (o [Hq, d],
    lse [Hq], weighted mean of |v| [Hq, d], largest sum of |q k| a row [Hq])."""
    hq, d = q.shape
    hkv, n, _ = k.shape
    if n == 0:
        z = np.zeros((hq, d))
        return z, np.full(hq, -np.inf), z, np.zeros(hq)
    qg = q.reshape(hkv, hq // hkv, d)
    s = np.einsum("hgd,hnd->hgn", qg, k) * scale
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    tot = p.sum(-1, keepdims=True)
    w = p / tot
    o = np.einsum("hgn,hnd->hgd", w, v).reshape(hq, d)
    wa = np.einsum("hgn,hnd->hgd", w, np.abs(v)).reshape(hq, d)
    big = (np.einsum("hgd,hnd->hgn", np.abs(qg), np.abs(k)) * scale).max(-1).reshape(hq)
    return o, (m + np.log(tot)).reshape(hq), wa, big
