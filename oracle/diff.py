"""Differential attention and the rotation by several axes, for the oracle (plain numpy in 64 bits,
from the definitions in include/attn.h).

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

from .cache import norm, pairs


def rotate_axes(x, cos_sin, positions, pair_axis, rot, interleaved):
    """Turns the pairs of x [tokens, rows, d] by the angles of positions [axes, tokens], pair i by
    axis pair_axis[i]."""
    y = np.array(x, dtype=np.float64)
    cs = np.asarray(cos_sin, dtype=np.float64)
    a, b = pairs(rot, interleaved) if rot else ((), ())
    for i, (p, q) in enumerate(zip(a, b)):
        at = np.asarray(positions)[pair_axis[i]]
        c, s = cs[at, i][:, None], cs[at, rot // 2 + i][:, None]
        first, second = y[..., p].copy(), y[..., q].copy()
        y[..., p] = first * c - second * s
        y[..., q] = second * c + first * s
    return y


def prepare(x, maps, weight, eps, cos_sin, positions, pair_axis, rot, interleaved):
    """Rows [tokens, heads, d], each of `maps` rows normed and turned apart. Returns (rows, the
    sizes |a| + |b| that the error of a turned channel goes by)."""
    t, h, d = x.shape
    x = np.asarray(x, np.float64).reshape(t, h * maps, d // maps)
    if weight is not None:
        x = norm(x, weight, eps)
    mag = np.abs(x)
    if rot:
        a, b = pairs(rot, interleaved)
        both = mag[..., a] + mag[..., b]
        mag[..., a], mag[..., b] = both, both
    y = rotate_axes(x, cos_sin, positions, pair_axis, rot, interleaved) if rot else x
    return y.reshape(t, h, d), mag.reshape(t, h, d)


def visible(mask, window, n):
    """Truth values [n, n] (row, key) of a dense mask, by name; 'document' masks are causal or full
    over their segments."""
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return {"none": np.ones((n, n), bool), "document_bidir": np.ones((n, n), bool),
            "causal": j <= i, "document": j <= i, "sliding": (j <= i) & (j > i - window),
            "sliding_bidir": np.abs(i - j) <= window, "prefix": (j <= i) | (j < window)}[mask]


class Rows:
    """Differential attention of q [Hq, n, d] over k, v [Hkv, m, d] (float64), here [n, m] truth
    values: o [Hq, n, d], lse [Hq, 2, n], and bounds on a kernel's error.

    Errors of a kernel that holds scores, sums and accumulators in 32 bits and rounds the softmax
    weights to `weight_step` (half a step, relative) and the output to bf16:
      * a score is off by at most e_m = 2^-18 max |q_m| |k_m| scale (64 products and their sums in
        fp32), so a weight by a factor exp(2 e_m) and its rounding: A_m v by
        E_m = (weight_step + expm1(2 e_m) + 2^-17) sum A_m |v|
        (2^-17: the exponentials' and the sums' own rounding);
      * y by E = E_1 + |lam| E_2; the root of mean y^2 by at most the root of mean E^2, the norm's
        quotient by (E + |y| rms(E) / rms) / (rms - rms(E)), rms with eps inside;
      * the output's rounding 2^-8 |o|; LSE_m by e_m + 2^-17 + 2^-22 |LSE_m|."""

    def __init__(self, q, k, v, here, lam, scale, weight, eps, out_scale, weight_step=2.0 ** -8):
        hq, n, d = q.shape
        g = hq // k.shape[0]
        half = d // 2
        y = np.zeros((hq, n, d))
        err = np.zeros((hq, n, d))
        self.lse = np.full((hq, 2, n), -np.inf)
        self.lse_tol = np.zeros((hq, 2, n))
        some = here.any(1)
        for h in range(hq):
            kk, vv = k[h // g], v[h // g]
            for m, f in ((0, 1.0), (1, -float(lam[h]))):
                if not kk.shape[0]:
                    continue
                cut = slice(m * half, (m + 1) * half)
                s = np.where(here, q[h][:, cut] @ kk[:, cut].T * scale, -np.inf)
                big = np.where(here, np.abs(q[h][:, cut]) @ np.abs(kk[:, cut]).T * scale, 0).max(1)
                top = np.where(some, s.max(1), 0.0)
                p = np.exp(s - top[:, None])
                tot = np.where(some, p.sum(1), 1.0)
                self.lse[h, m] = np.where(some, top + np.log(tot), -np.inf)
                w = p / tot[:, None]
                e = 2.0 ** -18 * big
                self.lse_tol[h, m] = e + 2.0 ** -17 + 2.0 ** -22 * np.where(
                    some, np.abs(self.lse[h, m]), 0)
                y[h] += f * (w @ vv)
                err[h] += abs(f) * (weight_step + np.expm1(2 * e) + 2.0 ** -17)[:, None] * (
                    w @ np.abs(vv))
        if weight is not None:
            rms = np.sqrt((y * y).mean(-1, keepdims=True) + eps)
            off = np.sqrt((err * err).mean(-1, keepdims=True))
            with np.errstate(divide="ignore", invalid="ignore"):
                low = np.where(rms > off, rms - off, 0.0)
                w = np.abs(np.asarray(weight, np.float64))
                err = np.where(some[:, None], (err + np.abs(y) * off / rms) / low * w, 0.0)
                y = np.where(some[:, None], y / rms * np.asarray(weight, np.float64), 0.0)
        self.o = out_scale * y
        self.o_tol = abs(out_scale) * err + 2.0 ** -8 * np.abs(self.o) + 1e-37


def two_norm(q, k, v, here, lam, scale, weight, eps, out_scale, weight_step=2.0 ** -8):
    """(o, bound [Hq, n]): Rows' o, and for every row a bound on the square of a kernel's error in
    2-norm, to be summed over many rows of a head.

    Roundings of different weights and outputs are independent of one another, so their squares add
    where Rows adds their sizes: with r = weight_step + 2 e_m + 2^-17 (Rows' relative error of one
    weight)
        E |dy_c|^2 <= r^2 sum_j (w_1j^2 + lam^2 w_2j^2) v_jc^2,
    the norm takes dy to at most |out_scale w_c dy_c| / rms (it drops the part along y), and the
    output's rounding adds (2^-8 o_c)^2. The bound takes each rounding at its largest; a rounding to
    bf16 is 0.43 of that in root mean square (uniform over a step, of mantissas from 1 to 2), so that
    the sum over a block of rows is about a fifth of the bound's."""
    rows = Rows(q, k, v, here, lam, scale, weight, eps, out_scale, weight_step)
    hq, n, d = q.shape
    g, half = hq // k.shape[0], d // 2
    bound = np.zeros((hq, n))
    some = here.any(1)
    for h in range(hq):
        kk, vv = k[h // g], v[h // g]
        y, var = np.zeros((n, d)), np.zeros((n, d))
        for m, f in ((0, 1.0), (1, -float(lam[h]))):
            cut = slice(m * half, (m + 1) * half)
            s = np.where(here, q[h][:, cut] @ kk[:, cut].T * scale, -np.inf)
            big = np.where(here, np.abs(q[h][:, cut]) @ np.abs(kk[:, cut]).T * scale, 0).max(1)
            w = np.exp(s - np.where(some, rows.lse[h, m], 0.0)[:, None])
            r = weight_step + 2.0 ** -17 * big + 2.0 ** -17
            y += f * (w @ vv)
            var += (f * r[:, None]) ** 2 * ((w * w) @ (vv * vv))
        if weight is not None:
            var *= (np.asarray(weight, np.float64)) ** 2 / ((y * y).mean(-1, keepdims=True) + eps)
        bound[h] = (out_scale * out_scale * var + (2.0 ** -8 * rows.o[h]) ** 2).sum(1)
    return rows.o, bound
