"""Differential attention at the edges of its numbers: rows whose squares leave fp32, scores of -inf.
Against plain 64-bit numpy, through the C ABI."""
import numpy as np
import pytest
import torch

from tiled_attention_gb300 import attn
from test_gpu_diff import (Chunk, Decode, Head, check, cuda_library, dev, diff, draw, f64,  # noqa: F401
                           run_diff, status)

pytestmark = pytest.mark.gpu


def scaled(tensors, values, amp):
    """bf16 tensors and their 64-bit values times powers of two by channel: exact."""
    amp = np.asarray(amp, np.float64)
    t = dev(amp.astype(np.float32)).to(torch.bfloat16) if amp.ndim else float(amp)
    return [x.mul_(t) for x in tensors], [v * amp for v in values]


def by_half(d, first, second):
    return np.repeat([first, second], d // 2)


def planes(h, o, lse, qv, kv, vv, mask, picks):
    """A few (batch, head) planes of dense attention against 64 bits."""
    lam, g = h.lam, qv.shape[1] // kv.shape[1]
    here = diff.visible(mask, 0, qv.shape[2])
    for b, x in picks:
        h.lam = lam[x:x + 1]
        check(f64(o[b, x:x + 1]), f64(lse[b, x:x + 1]),
              h.rows(qv[b, x:x + 1], kv[b, x // g:x // g + 1], vv[b, x // g:x // g + 1], here))
    h.lam = lam


# (B, Hq, Hkv, n, d): one CTA an SM at both head dims, and two at d = 64 with whole and shared tiles.
FORMS = [(1, 4, 2, 260, 64), (1, 4, 2, 260, 128), (12, 64, 4, 128, 64), (40, 64, 4, 17, 64)]
# Sizes of the values by half of the channels, and eps: squares that overflow or vanish in one half or
# both, on both sides of where they begin to, and those that eps outweighs.
SIZES = [(2.0 ** 100, 2.0 ** 100, 1e-5), (2.0 ** 66, 2.0 ** 66, 0.0), (2.0 ** 60, 2.0 ** 64, 1e-5),
         (2.0 ** 100, 1.0, 1e-5), (2.0 ** -60, 2.0 ** 90, 0.0), (2.0 ** -100, 2.0 ** -100, 0.0),
         (2.0 ** -47, 2.0 ** -53, 0.0), (2.0 ** -53, 2.0 ** -53, 1e-30), (1.0, 2.0 ** -60, 0.0),
         (2.0 ** -100, 2.0 ** -100, 1e-5), (2.0 ** -60, 2.0 ** -100, 1e-12)]


@pytest.mark.parametrize("B,Hq,Hkv,n,d", FORMS)
@pytest.mark.parametrize("first,second,eps", SIZES)
def test_norm_of_any_size(B, Hq, Hkv, n, d, first, second, eps):
    rng = np.random.default_rng(n + d)
    h = Head(rng, Hq, d, eps=eps)
    (q, qv), (k, kv), (v, vv) = (draw(rng, B, x, n, d) for x in (Hq, Hkv, Hkv))
    (v,), (vv,) = scaled([v], [vv], by_half(d, first, second))
    o, lse = run_diff(h, q, k, v, attn.ATTN_MASK_NONE)
    assert status() == 0
    planes(h, o, lse, qv, kv, vv, "none", [(0, 0), (B // 2, Hq // 2 + 1), (B - 1, Hq - 1)])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first,second,eps", SIZES)
def test_norm_of_any_size_over_pages(d, first, second, eps):
    """Chunks (at d = 64 with few and with many units) and single tokens, contexts of one worker and
    of several, up to 8 heads a kv head and more."""
    rng = np.random.default_rng(d)
    amp = by_half(d, first, second)
    for c in (Chunk(rng, [300, 40, 129], [150, 40, 1], 4, 2, d, 16),
              Chunk(rng, [150, 33, 277], [128, 33, 129], 64, 4, d, 32),
              Decode(rng, [1, 70, 5000, 20], 6, 2, d, 64), Decode(rng, [1, 3000], 24, 2, d, 16)):
        c.h.eps = eps
        scaled([c.v], [], amp)
        for x in c.ctx:
            x[1] *= amp
        out = c.run()
        assert status() == 0
        c.check(*(out or ()))


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_zero_are_zero(d):
    """y = 0 with eps = 0: o = 0 in every form."""
    rng = np.random.default_rng(d)
    for B, Hq, Hkv, n in ((1, 4, 2, 260), (40, 64, 4, 17)):
        h = Head(rng, Hq, d, eps=0.0)
        q, k, v = (draw(rng, B, x, n, d)[0] for x in (Hq, Hkv, Hkv))
        assert (run_diff(h, q, k, v.zero_(), attn.ATTN_MASK_CAUSAL)[0] == 0).all()
    c, w = Chunk(rng, [300, 40], [150, 1], 4, 2, d, 16), Decode(rng, [1, 5000, 0], 6, 2, d, 64)
    for x in (c, w):
        x.h.eps = 0.0
        x.v.nan_to_num_(0.0).zero_()
    assert (c.run()[0] == 0).all()
    w.run()
    assert status() == 0 and (w.o == 0).all()


# ------------------------------------------------------------------ scores of -inf
OUT = [(1, 4), (0, 1)]  # keys (first, every) out of a map's sight: some, all


def maps_apart(h, q, k, v, here, step):
    """(o, its bound, LSE [Hq, 2, n], its bound) where map m sees the keys here[m] [n, m] alone: y from
    oracle.diff.Rows of each map by itself, the norm and its bound as there."""
    half = q.shape[-1] // 2
    one = []
    for m in (0, 1):
        both = [np.concatenate([x[..., m * half:(m + 1) * half]] * 2, -1) for x in (q, k)]
        one.append(diff.Rows(*both, v, here[m], np.zeros_like(h.lam), h.scale, None, 0, 1.0, step))
    lam = h.lam.astype(np.float64)[:, None, None]
    y, err = one[0].o - lam * one[1].o, one[0].o_tol + np.abs(lam) * one[1].o_tol
    if h.weight is not None:
        rms, off = (np.sqrt((x * x).mean(-1, keepdims=True) + e) for x, e in ((y, h.eps), (err, 0.0)))
        low = np.where(rms > off, rms - off, 0.0)
        w = h.weight.astype(np.float64)
        with np.errstate(divide="ignore"):
            err = (err + np.abs(y) * off / rms) / low * np.abs(w)
        y = y / rms * w
    o = h.out_scale * y
    return (o, abs(h.out_scale) * err + 2.0 ** -8 * np.abs(o) + 1e-37,
            np.stack([x.lse[:, 0] for x in one], 1), np.stack([x.lse_tol[:, 0] for x in one], 1))


def check_apart(h, o, lse, q, k, v, here, step=2.0 ** -8):
    want, tol, want_lse, lse_tol = maps_apart(h, q, k, v, here, step)
    assert np.all(np.abs(o - want) <= tol), float(np.max(np.abs(o - want) - tol))
    dead = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), dead)
    assert np.all(np.abs(np.where(dead, 0, lse) - np.where(dead, 0, want_lse)) <= lse_tol)


def drown(q, qv, k, m, keys):
    """Scores of map m with `keys` (an index of k's rows) are -inf: a key channel of -inf against a
    query channel above zero."""
    at = m * q.shape[-1] // 2
    q[..., at], qv[..., at] = 1.0, 1.0
    k[keys + (at,)] = float("-inf")


def seen(here, m, first, every):
    """What each map sees where keys first, first + every, ... are out of map m's sight."""
    left = here & (np.arange(here.shape[1]) % every != first)
    return (left, here) if m == 0 else (here, left)


@pytest.mark.parametrize("m", [0, 1])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,n,d", FORMS)
@pytest.mark.parametrize("first,every", OUT)
def test_scores_of_minus_infinity(B, Hq, Hkv, n, d, normed, m, first, every):
    rng = np.random.default_rng(n + d + m)
    h = Head(rng, Hq, d, normed)
    (q, qv), (k, kv), (v, vv) = (draw(rng, B, x, n, d) for x in (Hq, Hkv, Hkv))
    drown(q, qv, k, m, (slice(None), slice(None), slice(first, None, every)))
    o, lse = run_diff(h, q, k, v, attn.ATTN_MASK_CAUSAL)
    assert status() == 0
    here = seen(diff.visible("causal", 0, n), m, first, every)
    for b in (0, B - 1):
        check_apart(h, f64(o[b]), f64(lse[b]), qv[b], kv[b], vv[b], here)


@pytest.mark.parametrize("m", [0, 1])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("d,Hq", [(64, 6), (128, 6), (64, 24), (128, 24)])
@pytest.mark.parametrize("first,every", OUT)
def test_scores_of_minus_infinity_over_pages(d, Hq, normed, m, first, every):
    rng = np.random.default_rng(d + Hq + m)
    c = Chunk(rng, [300, 40], [150, 1], Hq, 2, d, 16, normed)
    w = Decode(rng, [1, 70, 5000], Hq, 2, d, 64, normed)
    for x in (c, w):  # (pages hold multiples of `every` slots)
        drown(x.q, x.qv, x.k, m, (slice(None), slice(None), slice(first, None, every)))
    o, lse = c.run()
    w.run()
    assert status() == 0
    o, lse, at = f64(o[0]), f64(lse[0]), 0
    for b, (L, n) in enumerate(zip(c.lk, c.lq)):
        here = np.arange(L)[None] <= np.arange(L - n, L)[:, None]
        cut = slice(at, at + n)
        at += n
        check_apart(c.h, o[:, cut], lse[:, :, cut], c.qv[0][:, cut], *c.ctx[b], seen(here, m, first, every))
    for b, L in enumerate(w.lk):
        check_apart(w.h, f64(w.o[b]), f64(w.lse[b])[:, :, None], w.qv[b], *w.ctx[b],
                    seen(np.ones((1, L), bool), m, first, every), 2.0 ** -16)
