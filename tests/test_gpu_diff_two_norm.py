"""Differential attention's error in 2-norm over blocks of rows, against plain 64-bit numpy: an element's
worst case grows with the keys of its row, to a fifth of the output and more from 1400 keys on, and lets
a factor that is a few percent off pass; the 2-norm of a block does not. oracle.diff.two_norm derives the
bound; on these inputs it is below 2^-7 of the output, and test_two_norm_bounds_catch_small_mistakes
says what it catches."""
import numpy as np
import pytest

from test_gpu_diff import (KINDS, Chunk, Decode, Head, cuda_library, dev, diff, draw, f64,  # noqa: F401
                           run_diff, status)

pytestmark = pytest.mark.gpu


def check_norm(h, o, q, k, v, here, heads=None, step=2.0 ** -8):
    """o [Hq, n, d] of some heads, in blocks of 64 of a head's rows (the last one longer). Rows of under
    32 keys are left out: two maps over few keys may all but cancel."""
    g = q.shape[0] // k.shape[0]
    many = here.sum(1) >= 32
    o, q, here = o[:, many], q[:, many], here[many]
    for x in range(q.shape[0]) if heads is None else heads:
        want, bound = diff.two_norm(q[x:x + 1], k[x // g:x // g + 1], v[x // g:x // g + 1], here,
                                    h.lam[x:x + 1], h.scale, h.weight, h.eps, h.out_scale, step)
        err = ((o[x] - want[0]) ** 2).sum(1)
        size = (want[0] ** 2).sum(1)
        n = len(err)
        for a in range(0, max(1, n // 64)):
            cut = slice(64 * a, 64 * a + 64 if 64 * a + 128 <= n else n)
            assert bound[0, cut].sum() <= 2.0 ** -14 * size[cut].sum()
            assert err[cut].sum() <= bound[0, cut].sum(), (
                np.sqrt(err[cut].sum() / size[cut].sum()), np.sqrt(bound[0, cut].sum() / size[cut].sum()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("mask,window,B,Hq,Hkv,n", [("none", 0, 1, 4, 2, 1900), ("causal", 0, 1, 4, 1, 1399),
                                                    ("sliding", 500, 2, 24, 8, 1399),
                                                    ("sliding_bidir", 300, 1, 4, 4, 641),
                                                    ("none", 0, 4, 32, 4, 700),
                                                    ("none", 0, 12, 64, 4, 145)])
def test_dense_two_norm(mask, window, B, Hq, Hkv, n, d, normed):
    rng = np.random.default_rng(n + d + normed)
    h = Head(rng, Hq, d, normed)
    (q, qv), (k, kv), (v, vv) = (draw(rng, B, x, n, d) for x in (Hq, Hkv, Hkv))
    o, _ = run_diff(h, q, k, v, KINDS[mask], window)
    assert status() == 0
    here = diff.visible(mask, window, n)
    for b, heads in ((0, [0, Hq // 2 + 1]), (B - 1, [Hq - 1])):
        check_norm(h, f64(o[b]), qv[b], kv[b], vv[b], here, heads)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mask", ["document", "document_bidir"])
def test_document_two_norm(d, mask):
    rng = np.random.default_rng(d)
    lens = [1300, 200, 700]
    n, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    h = Head(rng, 8, d)
    (q, qv), (k, kv), (v, vv) = (draw(rng, 1, x, n, d) for x in (8, 2, 2))
    o, _ = run_diff(h, q, k, v, KINDS[mask], 0, dev(cu), len(lens))
    assert status() == 0
    o = f64(o[0])
    for a, b in zip(cu[:-1], cu[1:]):
        check_norm(h, o[:, a:b], qv[0][:, a:b], kv[0][:, a:b], vv[0][:, a:b],
                   diff.visible(mask, 0, b - a), [0, 5])


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("d,Hq,Hkv,many", [(64, 4, 2, False), (64, 64, 4, True), (128, 16, 4, False)])
def test_chunk_two_norm(d, page, Hq, Hkv, many):
    rng = np.random.default_rng(d + page)
    lk, lq = ([2100, 900, 1500], [64, 300, 17]) if not many else ([1000] * 6 + [1800], [70] * 6 + [300])
    c = Chunk(rng, lk, lq, Hq, Hkv, d, page)
    o, _ = c.run()
    assert status() == 0
    o, at = f64(o[0]), 0
    for b, (L, n) in enumerate(zip(lk, lq)):
        here = np.arange(L)[None] <= np.arange(L - n, L)[:, None]
        cut = slice(at, at + n)
        at += n
        if b in (0, len(lk) - 1):
            check_norm(c.h, o[:, cut], c.qv[0][:, cut], *c.ctx[b], here, [0, Hq - 1])


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 8, 2), (64, 24, 2), (128, 8, 2), (128, 16, 1)])
def test_decode_two_norm(d, Hq, Hkv):
    rng = np.random.default_rng(d + Hq)
    w = Decode(rng, [9000, 40, 700, 2500], Hq, Hkv, d, 64)
    w.run()
    assert status() == 0
    o = f64(w.o)
    for b, L in enumerate(w.lk):
        check_norm(w.h, o[b], w.qv[b], *w.ctx[b], np.ones((1, L), bool), step=2.0 ** -16)
