"""Differential prefill with many units a CTA whose rows do not go out by TMA (heads that share a tile,
segments' and chunks' last rows, a dense prompt's last tile): the shared memory that their rows were
normed in takes the Q of a later unit. Against plain 64-bit numpy, and the same bits each time."""
import numpy as np
import pytest
import torch

from tiled_attention_gb300 import attn
from test_gpu_diff import (KINDS, Chunk, Head, check, cuda_library, dev, diff, draw, f64,  # noqa: F401
                           run_diff, same_bits, status)

pytestmark = pytest.mark.gpu


def repeat(call, o, lse, times=8):
    for _ in range(times):
        o2, lse2 = call()
        assert same_bits(o, o2) and torch.equal(lse, lse2)


# At d = 64 more than four units an SM are two CTAs an SM, with several heads in the last tile (of 1,
# 17 and 64 rows) and a whole tile before it or none.
@pytest.mark.parametrize("B,Hq,Hkv,n,d", [(40, 64, 4, 17, 64), (12, 64, 4, 145, 64),
                                          (12, 64, 4, 129, 64), (24, 48, 8, 192, 64),
                                          (40, 64, 4, 17, 128), (16, 32, 8, 40, 128),
                                          (6, 32, 8, 300, 128), (24, 16, 16, 250, 64)])
@pytest.mark.parametrize("mask", ["none", "causal"])
def test_dense_rows_of_many_units(B, Hq, Hkv, n, d, mask):
    rng = np.random.default_rng(n + d)
    h = Head(rng, Hq, d)
    (q, qv), (k, kv), (v, vv) = (draw(rng, B, x, n, d) for x in (Hq, Hkv, Hkv))
    o, lse = run_diff(h, q, k, v, KINDS[mask])
    assert status() == 0
    here = diff.visible(mask, 0, n)
    for b in (0, B // 2, B - 1):
        check(f64(o[b]), f64(lse[b]), h.rows(qv[b], kv[b], vv[b], here))
    repeat(lambda: run_diff(h, q, k, v, KINDS[mask]), o, lse)
    assert status() == 0


@pytest.mark.parametrize("d,page,Hq,Hkv", [(64, 16, 64, 4), (64, 128, 24, 8), (128, 64, 32, 8),
                                           (128, 32, 16, 16)])
def test_chunk_rows_of_many_units(d, page, Hq, Hkv):
    rng = np.random.default_rng(d + page)
    lq = [int(x) for x in rng.integers(1, 17, 20)] + [40, 64, 65, 130, 200, 33]
    c = Chunk(rng, [n + int(x) for n, x in zip(lq, rng.integers(0, 400, len(lq)))], lq, Hq, Hkv, d,
              page)
    o, lse = c.run()
    assert status() == 0
    c.check(o, lse)
    repeat(c.run, o, lse)
    assert status() == 0


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 64, 4), (128, 32, 8)])
@pytest.mark.parametrize("mask", ["document", "document_bidir"])
def test_segment_rows_of_many_units(d, Hq, Hkv, mask):
    rng = np.random.default_rng(d)
    lens = [int(x) for x in rng.integers(1, 300, 25)]
    n, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    h = Head(rng, Hq, d)
    (q, qv), (k, kv), (v, vv) = (draw(rng, 1, x, n, d) for x in (Hq, Hkv, Hkv))
    call = lambda: run_diff(h, q, k, v, KINDS[mask], 0, dev(cu), len(lens))  # noqa: E731
    o, lse = call()
    assert status() == 0
    got, sums = f64(o[0]), f64(lse[0])
    for a, b in zip(cu[:-1], cu[1:]):
        check(got[:, a:b], sums[:, :, a:b], h.rows(qv[0][:, a:b], kv[0][:, a:b], vv[0][:, a:b],
                                                   diff.visible(mask, 0, b - a)))
    repeat(call, o, lse)
    assert status() == 0


def test_units_taken_over():
    """Thousands of units of uneven length, most of them taken over from blocks that have not begun
    (an answer and a request a unit and CTA), those without work among them: each row is written, and
    the same each time."""
    rng = np.random.default_rng(5)
    for d, Hq, Hkv in ((64, 64, 4), (128, 32, 8)):
        lens = [int(x) for x in rng.integers(0, 90, 60)] + [700, 0, 1300]
        n, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        h = Head(rng, Hq, d)
        (q, qv), (k, kv), (v, vv) = (draw(rng, 1, x, n, d) for x in (Hq, Hkv, Hkv))
        call = lambda: run_diff(h, q, k, v, attn.ATTN_MASK_DOCUMENT, 0, dev(cu),  # noqa: E731
                                len(lens))
        o, lse = call()
        assert status() == 0 and not torch.isnan(o).any() and not torch.isnan(lse).any()
        got, sums = f64(o[0]), f64(lse[0])
        for a, b in list(zip(cu[:-1], cu[1:]))[::7]:
            if a < b:
                check(got[:, a:b], sums[:, :, a:b], h.rows(qv[0][:, a:b], kv[0][:, a:b],
                                                           vv[0][:, a:b],
                                                           diff.visible("document", 0, b - a)))
        repeat(call, o, lse, 20)
        assert status() == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(96, 6), (64, 4), (24, 24)])
def test_chunks_of_one_and_two_ctas_an_sm(page, Hq, Hkv):
    """d = 64, on both sides of four tiles an SM (960, 640 and 240), tiles shared and not; a norm whose
    squares leave fp32 in some heads' values too."""
    rng = np.random.default_rng(page + Hq)
    for amp in (1.0, 2.0 ** 80):
        c = Chunk(rng, [900, 33, 777, 640, 128], [400, 33, 129, 1, 128], Hq, Hkv, 64, page)
        c.v[:, 0] *= amp
        for x in c.ctx:
            x[1, 0] *= amp
        o, lse = c.run()
        assert status() == 0
        c.check(o, lse)
        repeat(c.run, o, lse, 2)


@pytest.mark.parametrize("lens", [[64] * 3, [32] * 4, [64] * 5, [128, 30, 1], [17] * 30])
@pytest.mark.parametrize("d", [64, 128])
def test_few_documents(lens, d):
    """Documents whose tiles the GPU holds at once, and a few more."""
    rng = np.random.default_rng(len(lens) + d)
    n, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    h = Head(rng, 32, d)
    (q, qv), (k, kv), (v, vv) = (draw(rng, 1, x, n, d) for x in (32, 8, 8))
    for mask in ("document", "document_bidir"):
        o, lse = run_diff(h, q, k, v, KINDS[mask], 0, dev(cu), len(lens))
        assert status() == 0
        o, lse = f64(o[0]), f64(lse[0])
        for a, b in zip(cu[:-1], cu[1:]):
            check(o[:, a:b], lse[:, :, a:b], h.rows(qv[0][:, a:b], kv[0][:, a:b], vv[0][:, a:b],
                                                    diff.visible(mask, 0, b - a)))
