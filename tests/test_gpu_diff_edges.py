"""Differential attention at the edges of its numbers: rows whose squares leave fp32. Against plain
64-bit numpy, through the C ABI."""
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
