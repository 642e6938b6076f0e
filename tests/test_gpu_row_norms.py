"""Per-head norm of token rows whose squares leave fp32: norm and rotation, and appends to both caches,
by one and by several positions. A row times a power of two has the same norm with eps = 0, to the bit:
its sum of squares goes by an even power of two, and so does every step after it."""
import numpy as np
import pytest
import torch

from tiled_attention_gb300 import attn
from test_gpu_diff import (Pages, Proj, close, cuda_library, dev, f64, head_major, nan_like,  # noqa: F401
                           same_bits, status)

pytestmark = pytest.mark.gpu

POWERS = [100, 66, 63, -50, -54, -100]


def rows(r):
    """Outputs of every entry point that norms, for the projection r with eps = 0."""
    q, k, v = (r.part(x)[0] for x in "qkv")
    t, turn = r.total, list(r.turn())
    turn[2] = 0.0
    outs = []

    def out(h):
        outs.append(nan_like(1, h, t, r.d))
        return outs[-1]

    attn.check(attn.attn_norm_rope_axes(q, k, out(r.Hq), out(r.Hkv), t, t, r.Hq, r.Hkv, r.d, r.maps,
                                        r.width, r.width, *turn))
    page, num = 16, -(-t // 16)
    table = dev(np.arange(num, dtype=np.int32)[None])
    cu, lk = dev(np.array([0, t], np.int32)), dev(np.array([t], np.int32))

    def pools(width):
        outs.extend(torch.zeros((num, r.Hkv, page, width), dtype=torch.int16, device="cuda")
                    for _ in range(2))
        return outs[-2:]

    attn.check(attn.attn_append_paged_axes(q, k, v, out(r.Hq), *pools(r.d), 1, r.Hq, r.Hkv, t, t, r.d,
                                           r.maps, r.width, r.width, r.width, *turn, cu, lk, table, num,
                                           page, num))
    if r.maps == 1:
        one = turn[:7]
        attn.check(attn.attn_norm_rope(q, k, out(r.Hq), out(r.Hkv), t, t, r.Hq, r.Hkv, r.d, r.width,
                                       r.width, *one, r.d_pos[0].contiguous()))
        args = (1, r.Hq, r.Hkv, t, t, r.d, r.width, r.width, r.width)
        attn.check(attn.attn_append_paged(q, k, v, out(r.Hq), *pools(r.d), *args, *one, cu, lk, table,
                                          num, page, num))
        attn.check(attn.attn_append_paged_fp4(q, k, v, out(r.Hq), *pools(r.d * 9 // 32), 0.01, 0.01,
                                              *args, *one, cu, lk, table, num, page, num))
        outs[-1] = None  # values of 4 bits are not normed
    assert status() == 0
    return [o.view(torch.int16) for o in outs if o is not None]


@pytest.mark.parametrize("d,maps", [(64, 1), (128, 1), (64, 2), (128, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens", [7, 6000])
def test_norm_does_not_go_by_a_power_of_two(d, maps, interleaved, tokens):
    """One warp a row group and one warp a token; rows of all sizes in one warp too."""
    rng = np.random.default_rng(d + maps)
    r = Proj(rng, tokens, 5, 3, d, maps, d // maps // 2, 2, "turns", interleaved, True,
             max_pos=tokens)
    hk = (r.Hq + r.Hkv) * d  # queries and keys
    # x 2^-100 is x again in bf16 only from |x| = 2^-26 on (its least normal number is 2^-126); one of
    # these six million values lies at 2^-27.3 and came back as another.
    r.buf[r.buf.abs() < 2.0 ** -26] = 0
    was = r.buf.clone()
    want = rows(r)
    for p in POWERS:
        r.buf.copy_(was)
        r.buf[:, :hk] *= 2.0 ** p
        for a, b in zip(rows(r), want):
            assert torch.equal(a, b)
    heads = torch.tensor([2.0 ** p for p in (0, 90, -90, 65, -60, 0, 100, -30)], device="cuda")
    r.buf.copy_(was)
    r.buf[:, :hk] *= heads.repeat_interleave(d).to(torch.bfloat16)
    for a, b in zip(rows(r), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,maps", [(64, 1), (128, 2)])
@pytest.mark.parametrize("power", [100, 64, 0, -30])
def test_norm_against_64_bits(d, maps, power):
    """With eps = 1e-5, where small rows go by eps."""
    rng = np.random.default_rng(d)
    r = Proj(rng, 30, 6, 2, d, maps, 32, 3, "any", norm=True)
    r.buf *= 2.0 ** power
    r.x = r.x * 2.0 ** power
    qo, ko = r.norm_rope(r.total)
    assert status() == 0
    for name, got in (("q", qo), ("k", ko)):
        want, mag = r.want(name)
        close(f64(got), head_major(want, r.total), head_major(mag, r.total))


def test_rows_of_zero_are_zero():
    """With eps = 0, of either sign (a turn takes zeros times cosines below zero): bf16 bits, and at
    the end those of 4-bit keys."""
    r = Proj(np.random.default_rng(1), 40, 4, 2, 128, 1, 64, 2, "turns", norm=True)
    r.buf.zero_()
    *outs, codes = rows(r)
    for x in outs:
        assert (x & 0x7FFF == 0).all()
    assert (codes & 0x7777 == 0).all()
