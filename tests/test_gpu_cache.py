"""Norm and rotation, paged append in bf16 and 4 bits, 4-bit pages back to bf16 and the 4-bit
paged decode, against plain 64-bit numpy, through the C ABI.

Tolerances:
  * a bf16 result is off by half a step, 2^-8 of its value, plus the fp32 arithmetic's error,
    here bounded by 2^-19 of the pair's (|a| + |b|): the norm's sum of 128 squares over 8
    lanes (16 fused adds and 3 shuffled ones, halved by the root), its reciprocal root (2 ulp)
    and products come to less than 18 * 2^-24, a turn's three roundings to 3 * 2^-24;
  * 4-bit codes and scales of un-normed keys and of values equal the definition's byte for byte
    (every step is an IEEE fp32 operation); normed keys, whose rsqrt may differ in the last bits,
    are within one code step;
  * decode: bf16 output 2^-8 |O|; softmax weights rounded to f16, 2^-11 of the weighted mean of
    |v|, and as much again for scores off by up to 2^-18 sum |q k| (128 products accumulated in
    fp32 by 8 MMAs) with sum |q k| up to 2^6; f16 weights below 2^-14 lose up to 2^-25 each
    against a largest weight of at least 2^7, over 2^14 keys 2^-18 max |v|.
    LSE: the scores' error, 2^-17 for the sums, 2^-22 of its value.
Outputs are pre-filled so that a row the kernels never write fails loudly."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache
from tiled_attention_gb300 import attn
from tiled_attention_gb300 import inputs as I
from tiled_attention_gb300.runner import bf16_tensor

pytestmark = pytest.mark.gpu

EPS = 1e-6
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tiled_attention_gb300 import build
    build.build()
    attn.lib()
    torch.cuda.synchronize()
    assert attn.attn_get_status() == 0


def status():
    torch.cuda.synchronize()
    return attn.attn_get_status()


def dev(a, dtype=None):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a if dtype is None else a.astype(dtype)).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def table_of(rng, max_pos, rot):
    """A cos / sin table of arbitrary angles, fp32."""
    ang = rng.uniform(-np.pi, np.pi, (max_pos, rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


class Rows:
    """A projection's token rows (q | k | v), norm weights and a rotation table."""

    def __init__(self, rng, total, Hq, Hkv, d, rot, max_pos=64, interleaved=False, norm=False,
                 pad=0, amp=1.0):
        self.total, self.Hq, self.Hkv, self.d = total, Hq, Hkv, d
        self.rot, self.interleaved, self.max_pos = rot, interleaved, max_pos
        self.width = (Hq + 2 * Hkv) * d + pad
        x = rng.standard_normal((total, self.width)).astype(np.float32) * np.float32(amp)
        self.bits = I.f32_to_bf16_bits(x)
        self.x = I.bf16_bits_to_f32(self.bits).astype(np.float64)
        self.buf = bf16_tensor(self.bits, "cuda")
        self.cs = table_of(rng, max_pos, max(rot, 2))[:, :max(rot, 2)]
        self.cos_sin = dev(self.cs) if rot else None
        w = (1 + 0.3 * rng.standard_normal((2, d))).astype(np.float32)
        self.w = [w[0], w[1]] if norm else [None, None]
        self.weights = [None if a is None else dev(a) for a in self.w]

    def part(self, name):
        lo = {"q": 0, "k": self.Hq, "v": self.Hq + self.Hkv}[name]
        h = self.Hq if name == "q" else self.Hkv
        sl = slice(lo * self.d, (lo + h) * self.d)
        return self.buf[:, sl], self.x[:, sl].reshape(-1, h, self.d)

    def want(self, name, pos):
        """(prepared rows, error scale |a| + |b|), float64 [total, H, d]."""
        x = self.part(name)[1]
        w = self.w[0 if name == "q" else 1]
        if w is not None:
            x = cache.norm(x, w, EPS)
        mag = np.abs(x)
        if self.rot:
            a, b = cache.pairs(self.rot, self.interleaved)
            both = mag[..., a] + mag[..., b]
            mag = mag.copy()
            mag[..., a] = both
            mag[..., b] = both
        return cache.rotate(x, self.cs, pos, self.rot, self.interleaved), mag


def close(got, want, mag):
    err = np.abs(got - want)
    tol = BF16_HALF * np.abs(want) + 2.0 ** -19 * mag
    assert np.all(err <= tol), float(np.max(err - tol))


def head_major(x, N):
    t, h, d = x.shape
    return x.reshape(t // N, N, h, d).transpose(0, 2, 1, 3)


# ------------------------------------------------------------------ norm and rotation

def run_norm_rope(r, N, positions=None, q=True, k=True):
    qo = torch.full((r.total // N, r.Hq, N, r.d), float("nan"), dtype=torch.bfloat16,
                    device="cuda")
    ko = torch.full((r.total // N, r.Hkv, N, r.d), float("nan"), dtype=torch.bfloat16,
                    device="cuda")
    rc = attn.attn_norm_rope(r.part("q")[0] if q else None, r.part("k")[0] if k else None,
                             qo if q else None, ko if k else None, r.total, N, r.Hq, r.Hkv, r.d,
                             r.width, r.width, r.weights[0], r.weights[1], EPS, r.cos_sin,
                             r.max_pos if r.rot else 0, r.rot, r.interleaved,
                             None if positions is None else dev(positions, np.int32))
    assert rc == 0, attn.last_error()
    return qo, ko


@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 0), (128, 16),
                                   (128, 80), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope(d, rot, interleaved, norm):
    rng = np.random.default_rng(d + rot + 2 * interleaved + norm)
    for total, N, Hq, Hkv, pad in ((1, 1, 1, 1, 0), (6, 3, 5, 3, 8), (35, 7, 32, 8, 0),
                                   (61, 61, 9, 2, 24)):
        r = Rows(rng, total, Hq, Hkv, d, rot, interleaved=interleaved, norm=norm, pad=pad)
        pos = rng.integers(0, r.max_pos, total)
        for given in (True, False):
            p = pos if given else np.arange(total) % N
            qo, ko = run_norm_rope(r, N, pos if given else None)
            assert status() == 0
            for name, got in (("q", qo), ("k", ko)):
                want, mag = r.want(name, p)
                close(f64(got), head_major(want, N), head_major(mag, N))


def test_norm_rope_one_tensor_alone():
    rng = np.random.default_rng(5)
    r = Rows(rng, 10, 4, 2, 128, 128, norm=True)
    both = run_norm_rope(r, 5)
    assert torch.equal(run_norm_rope(r, 5, k=False)[0].view(torch.int16),
                       both[0].view(torch.int16))
    assert torch.equal(run_norm_rope(r, 5, q=False)[1].view(torch.int16),
                       both[1].view(torch.int16))


def test_norm_rope_many_tokens():
    """Enough tokens for one warp a token; split and unsplit rows agree bit for bit."""
    rng = np.random.default_rng(6)
    r = Rows(rng, 5003, 12, 3, 64, 64, max_pos=6000, norm=True)
    pos = rng.integers(0, 6000, r.total)
    qo, ko = run_norm_rope(r, r.total, pos)
    want, mag = r.want("q", pos)
    close(f64(qo), head_major(want, r.total), head_major(mag, r.total))
    few = Rows(np.random.default_rng(6), 5003, 12, 3, 64, 64, max_pos=6000, norm=True)
    few.total, few.buf = 40, few.buf[:40]
    q2, k2 = run_norm_rope(few, 40, pos[:40])
    assert torch.equal(q2[0].view(torch.int16), qo[0, :, :40].contiguous().view(torch.int16))
    assert torch.equal(k2[0].view(torch.int16), ko[0, :, :40].contiguous().view(torch.int16))


def test_norm_rope_bad_position_leaves_its_rows():
    rng = np.random.default_rng(7)
    r = Rows(rng, 6, 2, 1, 128, 64, max_pos=10)
    pos = np.array([3, 10, 0, -1, 9, 2 ** 31 - 1])
    qo, ko = run_norm_rope(r, 1, pos)
    assert status() == attn.ATTN_ERR_BOUNDS
    good = np.array([0, 2, 4])
    assert torch.isnan(qo[[1, 3, 5]]).all() and torch.isnan(ko[[1, 3, 5]]).all()
    want, mag = r.want("q", np.clip(pos, 0, 9))
    close(f64(qo)[good, :, 0], want[good], mag[good])


def test_norm_rope_extreme_rows():
    """Zero rows stay zero under the norm, rows of the type's largest values saturate nothing
    that 64 bits do not, and a row of NaN stays its own."""
    rng = np.random.default_rng(8)
    r = Rows(rng, 4, 2, 1, 128, 128, norm=True)
    x = r.buf.clone()
    x[0] = 0
    x[1] = float("nan")
    r.buf = x
    r.x = f64(x)
    pos = np.array([1, 2, 3, 4])
    qo, ko = run_norm_rope(r, 1, pos)
    assert (qo[0] == 0).all() and torch.isnan(qo[1]).all()
    want, mag = r.want("q", pos)
    close(f64(qo)[2:, :, 0], want[2:], mag[2:])


# ------------------------------------------------------------------ append

class Batch:
    """Sequences of lq new tokens at the end of contexts lk, in a shuffled page pool."""

    def __init__(self, rng, lk, lq, page, spare=5, behind=0):
        self.lk, self.lq, self.page = np.asarray(lk), np.asarray(lq), page
        per = -(-self.lk // page)
        self.num = int(per.sum()) + spare
        perm = rng.permutation(self.num)
        self.cols = max(1, int(per.max()))
        self.table = np.full((len(lk), self.cols), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(self.lq)]).astype(np.int32)
        self.real = int(self.cu[-1])
        self.total = self.real + behind
        pos, phys, slot = [], [], []
        for b in range(len(lk)):
            p = np.arange(self.lk[b] - self.lq[b], self.lk[b])
            f, s = cache.slots(p, self.table[b], page)
            pos.append(p), phys.append(f), slot.append(s)
        self.pos = np.concatenate(pos + [np.zeros(behind, int)]).astype(int)
        self.phys, self.slot = np.concatenate(phys).astype(int), np.concatenate(slot).astype(int)
        self.d_cu, self.d_lk = dev(self.cu), dev(self.lk, np.int32)
        self.d_table = dev(self.table)

    def args(self):
        return (self.d_cu, self.d_lk, self.d_table, self.cols, self.page, self.num)


def row_args(r):
    return (r.width, r.width, r.width, r.weights[0], r.weights[1], EPS, r.cos_sin,
            r.max_pos if r.rot else 0, r.rot, r.interleaved)


def pools_bf16(rng, bt, Hkv, d):
    bits = I.normal_bf16(rng, (2, bt.num, Hkv, bt.page, d))
    return bits, bf16_tensor(bits[0], "cuda"), bf16_tensor(bits[1], "cuda")


def append_bf16(r, bt, kp, vp, N, q=True):
    qo = torch.full((bt.total // N, r.Hq, N, r.d), float("nan"), dtype=torch.bfloat16,
                    device="cuda")
    rc = attn.attn_append_paged(r.part("q")[0] if q else None, r.part("k")[0], r.part("v")[0],
                                qo if q else None, kp, vp, len(bt.lk), r.Hq, r.Hkv, bt.total, N,
                                r.d, *row_args(r), *bt.args())
    assert rc == 0, attn.last_error()
    return qo


RAGGED = [([1], [1]), ([40, 7, 0, 129, 16], [3, 7, 0, 1, 16]), ([65, 64, 63, 128], [1, 1, 1, 1]),
          ([300, 1, 48], [210, 1, 33])]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,rot,interleaved,norm", [(64, 16, False, True), (64, 64, True, False),
                                                    (128, 128, False, True), (128, 0, False, False),
                                                    (128, 48, True, True)])
def test_append_paged(page, d, rot, interleaved, norm):
    rng = np.random.default_rng(page + d + rot)
    for (lk, lq), behind, (Hq, Hkv) in zip(RAGGED, (0, 3, 0, 2), ((4, 4), (6, 2), (8, 1), (5, 5))):
        bt = Batch(rng, lk, lq, page, behind=behind)
        r = Rows(rng, bt.total, Hq, Hkv, d, rot, max_pos=320, interleaved=interleaved, norm=norm)
        bits, kp, vp = pools_bf16(rng, bt, Hkv, d)
        N = 1 if max(lq) == 1 else bt.total
        qo = append_bf16(r, bt, kp, vp, N)
        assert status() == 0
        want, mag = r.want("q", bt.pos)
        got = f64(qo)
        n = bt.real
        tok = got.transpose(0, 2, 1, 3).reshape(bt.total, Hq, d)
        close(tok[:n], want[:n], mag[:n])
        assert np.isnan(tok[n:]).all(), "rows behind the last sequence were written"
        kgot, vgot = f64(kp), f64(vp)
        want, mag = r.want("k", bt.pos)
        close(kgot[bt.phys, :, bt.slot], want[:n], mag[:n])
        assert np.array_equal(vgot[bt.phys, :, bt.slot], r.part("v")[1][:n])
        # every other slot as it was
        old = I.bf16_bits_to_f32(bits).astype(np.float64)
        for got, was in ((kgot, old[0]), (vgot, old[1])):
            got[bt.phys, :, bt.slot] = was[bt.phys, :, bt.slot]
            assert np.array_equal(got, was)


def test_append_without_queries():
    rng = np.random.default_rng(11)
    bt = Batch(rng, [50, 20], [30, 1], 16)
    r = Rows(rng, bt.total, 4, 2, 128, 128, max_pos=64, norm=True)
    _, kp, vp = pools_bf16(rng, bt, 2, 128)
    k2, v2 = kp.clone(), vp.clone()
    append_bf16(r, bt, kp, vp, bt.total)
    append_bf16(r, bt, k2, v2, bt.total, q=False)
    assert torch.equal(kp.view(torch.int16), k2.view(torch.int16))
    assert torch.equal(vp.view(torch.int16), v2.view(torch.int16))


def test_append_many_sequences():
    """More sequences than a warp has lanes, empty ones among them: the search for a token's
    sequence."""
    rng = np.random.default_rng(12)
    lk = rng.integers(1, 40, 1500)
    lq = np.minimum(rng.integers(0, 3, 1500), lk)
    bt = Batch(rng, lk, lq, 16, behind=9)
    r = Rows(rng, bt.total, 1, 1, 64, 64, max_pos=40)
    _, kp, vp = pools_bf16(rng, bt, 1, 64)
    append_bf16(r, bt, kp, vp, bt.total)
    assert status() == 0
    want, mag = r.want("k", bt.pos)
    close(f64(kp)[bt.phys, :, bt.slot], want[:bt.real], mag[:bt.real])
    assert np.array_equal(f64(vp)[bt.phys, :, bt.slot], r.part("v")[1][:bt.real])


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("fault", ["long", "short", "decreasing", "start", "past", "page",
                                   "negative page", "position"])
def test_append_device_checks(fp4, fault):
    """Bad lengths, pages and positions are reported and never written through; the other
    sequences' tokens are."""
    rng = np.random.default_rng(13)
    bt = Batch(rng, [40, 20, 33], [5, 2, 4], 16)
    r = Rows(rng, bt.total, 2, 2, 128, 128, max_pos=40)
    cu, lk, table = bt.cu.copy(), bt.lk.astype(np.int32), bt.table.copy()
    code, hurt = attn.ATTN_ERR_SEQLENS, [1]
    if fault == "long":
        lk[1] = bt.cols * 16 + 1
    elif fault == "short":
        lk[1] = 1
    elif fault == "decreasing":
        cu[2] = 3
        hurt = [0, 1, 2]  # which tokens whose sequence is found varies: none is checked
    elif fault == "start":
        cu[0] = -1
        hurt = [0]
    elif fault == "past":
        cu[3] = bt.total + 1
        hurt = [2]
    elif fault == "page":
        table[1, 1] = bt.num
        code = attn.ATTN_ERR_BOUNDS
    elif fault == "negative page":
        table[1, 1] = -7
        code = attn.ATTN_ERR_BOUNDS
    else:
        r.max_pos = 39  # the last token of sequence 0
        code, hurt = attn.ATTN_ERR_BOUNDS, [0]
    bt.d_cu, bt.d_lk, bt.d_table = dev(cu), dev(lk), dev(table)
    if fp4:
        kp, vp = (torch.zeros((bt.num, 2, 16 * 72), dtype=torch.uint8, device="cuda")
                  for _ in range(2))
        append_fp4(r, bt, kp, vp, bt.total, 1.0, 1.0)
        codes, sf = cache.split_block(vp.cpu().numpy(), 16, 128)
        vgot = cache.values(codes, sf, 1.0)
        vwant = cache.values(*cache.quantize(r.part("v")[1].astype(np.float32), 1.0), 1.0)
    else:
        kp, vp = (torch.zeros((bt.num, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))
        append_bf16(r, bt, kp, vp, bt.total)
        vgot, vwant = f64(vp), r.part("v")[1]
    assert status() == code
    for b in range(3):
        if b in hurt:
            continue
        sl = slice(bt.cu[b], bt.cu[b + 1])
        assert np.array_equal(vgot[bt.phys[sl], :, bt.slot[sl]], vwant[sl])
    if fault in ("long", "short", "page", "negative page", "position"):
        sl = slice(bt.cu[hurt[0]], bt.cu[hurt[0] + 1])
        wrong = vgot[bt.phys[sl], :, bt.slot[sl]]
        if fault == "position":  # the other tokens of that sequence are fine
            assert not wrong[-1].any() and np.array_equal(wrong[:-1], vwant[sl][:-1])
        elif "page" in fault:  # one of its two tokens sits on the good page 1 or both do
            on = bt.pos[sl] // 16 == 1
            assert not wrong[on].any() and np.array_equal(wrong[~on], vwant[sl][~on])
        else:
            assert not wrong.any()
    elif fault in ("start", "past"):  # nothing of the sequence anywhere: zeros but the others'
        keep = np.concatenate([np.arange(bt.cu[b], bt.cu[b + 1]) for b in range(3)
                               if b not in hurt])
        vgot[bt.phys[keep], :, bt.slot[keep]] = 0
        assert not vgot.any()


# ------------------------------------------------------------------ append in 4 bits

def append_fp4(r, bt, kp, vp, N, ks, vs, q=True):
    qo = torch.full((bt.total // N, r.Hq, N, r.d), float("nan"), dtype=torch.bfloat16,
                    device="cuda")
    rc = attn.attn_append_paged_fp4(r.part("q")[0] if q else None, r.part("k")[0],
                                    r.part("v")[0], qo if q else None, kp, vp, ks, vs,
                                    len(bt.lk), r.Hq, r.Hkv, bt.total, N, r.d, *row_args(r),
                                    *bt.args())
    assert rc == 0, attn.last_error()
    return qo


def pools_fp4(rng, num, Hkv, page, d):
    return [torch.from_numpy(rng.integers(0, 256, (num, Hkv, page * (d // 2 + d // 16)),
                                          dtype=np.uint8)).cuda() for _ in range(2)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 32, False), (64, 64, False), (64, 16, True),
                                               (128, 96, False), (128, 128, False), (128, 0, False),
                                               (128, 112, True)])
def test_append_fp4_bytes(page, d, rot, interleaved):
    rng = np.random.default_rng(100 + page + d + rot)
    for (lk, lq), behind, (Hq, Hkv) in zip(RAGGED, (0, 3, 0, 2), ((4, 4), (6, 2), (8, 1), (5, 5))):
        bt = Batch(rng, lk, lq, page, behind=behind)
        r = Rows(rng, bt.total, Hq, Hkv, d, rot, max_pos=320, interleaved=interleaved,
                 amp=float(np.exp(rng.uniform(-3, 5))))
        kp, vp = pools_fp4(rng, bt.num, Hkv, page, d)
        old = [kp.cpu().numpy(), vp.cpu().numpy()]
        ks, vs = 0.3, 2.0 ** -5
        N = 1 if max(lq) == 1 else bt.total
        qo = append_fp4(r, bt, kp, vp, N, ks, vs)
        assert status() == 0
        n = bt.real
        want, mag = r.want("q", bt.pos)
        tok = f64(qo).transpose(0, 2, 1, 3).reshape(bt.total, Hq, d)
        close(tok[:n], want[:n], mag[:n])
        assert np.isnan(tok[n:]).all()
        k32 = cache.rotate(r.part("k")[1], r.cs, bt.pos, rot, interleaved, np.float32)
        for pool, was, rows, scale in ((kp, old[0], k32, ks), (vp, old[1], r.part("v")[1], vs)):
            codes, sf = cache.quantize(rows[:n].astype(np.float32), scale)
            wc, ws = (a.copy() for a in cache.split_block(was, page, d))
            wc[bt.phys, :, bt.slot] = codes
            ws[bt.phys, :, bt.slot] = sf
            gc, gs = cache.split_block(pool.cpu().numpy(), page, d)
            assert np.array_equal(gs, ws)
            assert np.array_equal(gc, wc)


def test_append_fp4_edges():
    """All-zero blocks, blocks whose scale rounds to zero or to a subnormal, saturating ones,
    values on the codes' midpoints, negative zeros: byte for byte."""
    rng = np.random.default_rng(101)
    bt = Batch(rng, [16], [16], 16)
    r = Rows(rng, 16, 1, 2, 128, 0)
    x = np.array(r.x, np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= np.float32(2.0 ** -14)
    x[3] *= np.float32(2.0 ** -9)
    x[4] *= np.float32(3e4)
    x[5] *= np.float32(1e30)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2)
    x[6] = np.tile(np.concatenate([mids[:8], -mids[:8]]), x.shape[1] // 16)
    x[7] = x[6] * 8
    x[8, ::16] = 448 * 6
    x[9, ::2] = -0.0
    x[10] = np.float32(1e-38)
    bits = I.f32_to_bf16_bits(x)
    r.x = I.bf16_bits_to_f32(bits).astype(np.float64)
    r.buf = bf16_tensor(bits, "cuda")
    for ks, vs in ((1.0, 1.0), (0.013, 7.0)):
        kp, vp = pools_fp4(rng, bt.num, 2, 16, 128)
        append_fp4(r, bt, kp, vp, 16, ks, vs, q=False)
        assert status() == 0
        for pool, name, scale in ((kp, "k", ks), (vp, "v", vs)):
            codes, sf = cache.quantize(r.part(name)[1].astype(np.float32), scale)
            gc, gs = cache.split_block(pool.cpu().numpy(), 16, 128)
            assert np.array_equal(gs[bt.phys, :, bt.slot], sf)
            assert np.array_equal(gc[bt.phys, :, bt.slot], codes)


@pytest.mark.parametrize("d,rot,interleaved", [(64, 32, False), (128, 0, False), (128, 64, True),
                                               (128, 128, False)])
def test_append_fp4_infinities_and_nan(d, rot, interleaved):
    """Infinite values, and finite ones whose quotient by the tensor scale overflows, saturate:
    scale 448, codes of 6. A NaN makes its own block's scale NaN and its codes zero."""
    rng = np.random.default_rng(104)
    bt = Batch(rng, [16], [16], 16)
    r = Rows(rng, 16, 1, 2, d, rot, interleaved=interleaved)
    x = np.array(r.x, np.float32)
    inf, nan = np.float32(np.inf), np.float32(np.nan)
    x[1, 5::40] = inf
    x[2, 3::24] = -inf
    x[3] = np.where(np.arange(x.shape[1]) % 2, inf, -inf)
    x[4] = np.float32(3e38) * np.sign(x[4])
    x[5, ::37] = np.float32(-2e38)
    x[6, 9::50] = nan
    x[7] = nan
    x[8, 4::48], x[8, 20::48] = inf, nan
    x[9, ::8] = np.float32(4200.0)
    bits = I.f32_to_bf16_bits(np.where(np.isfinite(x), x, 0).astype(np.float32))
    top = (np.ascontiguousarray(x).view(np.uint32) >> 16).astype(np.uint16)
    bits = np.where(np.isfinite(x), bits, top)
    r.x = I.bf16_bits_to_f32(bits).astype(np.float64)
    r.buf = bf16_tensor(bits, "cuda")
    for ks, vs in ((1.0, 1.0), (0.003, 2.0 ** -20)):
        kp, vp = pools_fp4(rng, bt.num, 2, 16, d)
        append_fp4(r, bt, kp, vp, 16, ks, vs, q=False)
        assert status() == 0
        with np.errstate(all="ignore"):
            k32 = cache.rotate(r.part("k")[1], r.cs, bt.pos, rot, interleaved, np.float32)
        for pool, rows, scale in ((kp, k32, ks), (vp, r.part("v")[1], vs)):
            y = rows.astype(np.float32)
            with np.errstate(over="ignore"):
                xs = y * (np.float32(1) / np.float32(scale))
            lost = np.isnan(xs.reshape(16, 2, d // 16, 16)).any(-1)
            y = np.where(np.repeat(lost, 16, -1), np.float32(0), y)
            with np.errstate(all="ignore"):
                codes, sf = cache.quantize(y, scale)
            assert lost[6:9].any() and not lost[1].all() and (sf == 0x7E).any()
            sf[lost] = 0x7F
            gc, gs = cache.split_block(pool.cpu().numpy(), 16, d)
            assert np.array_equal(gs[bt.phys, :, bt.slot], sf)
            assert np.array_equal(gc[bt.phys, :, bt.slot], codes)


def test_append_fp4_normed_within_a_step():
    """|value - y| is at most half the widest step (1 * scale, or 0.4 * scale where 6 saturates),
    the scale at most max |y| / 6 * (1 + 2^-4)."""
    rng = np.random.default_rng(102)
    bt = Batch(rng, [90, 33], [90, 20], 32)
    r = Rows(rng, bt.total, 2, 2, 128, 128, max_pos=90, norm=True)
    kp, vp = pools_fp4(rng, bt.num, 2, 32, 128)
    append_fp4(r, bt, kp, vp, bt.total, 0.01, 1.0)
    assert status() == 0
    codes, sf = cache.split_block(kp.cpu().numpy(), 32, 128)
    got = cache.values(codes, sf, 0.01)[bt.phys, :, bt.slot]
    want, _ = r.want("k", bt.pos)
    top = np.abs(want).reshape(*want.shape[:-1], -1, 16).max(-1).repeat(16, axis=-1)
    assert np.all(np.abs(got - want) <= top / 6 * (1 + 2.0 ** -4) + 1e-6)


# ------------------------------------------------------------------ unpack

@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,Hkv", [(64, 1), (64, 5), (128, 2)])
def test_unpack(page, d, Hkv):
    rng = np.random.default_rng(200 + page + d)
    bt = Batch(rng, [1, page, 0, 3 * page + 7, page - 1], [0] * 5, page)
    pool, _ = pools_fp4(rng, bt.num, Hkv, page, d)  # any byte, NaN scales among them
    codes, sf = cache.split_block(pool.cpu().numpy(), page, d)
    ok = (sf & 0x7F) != 0x7F
    sf = np.where(ok, sf, 0x38).astype(np.uint8)
    lens = bt.lk.copy()
    raw = pool.cpu().numpy()
    # finite scales in valid slots, NaN ones left past the lengths
    cut = page * d // 2
    fixed = raw.copy().reshape(bt.num, Hkv, -1)
    tail = fixed[:, :, cut:].reshape(bt.num, Hkv, page, d // 16)
    bad = np.full_like(tail, 0x7F)
    for b in range(5):
        f, s = cache.slots(np.arange(lens[b]), bt.table[b], page)
        bad[f, :, s] = sf[f, :, s]
    fixed[:, :, cut:] = bad.reshape(bt.num, Hkv, -1)
    dst = torch.full((5 * bt.cols, Hkv, page, d), 7.0, dtype=torch.bfloat16, device="cuda")
    scale = 0.37
    rc = attn.attn_unpack_pages_fp4(dev(fixed), dst, scale, bt.d_table, bt.d_lk, 5, bt.cols, Hkv,
                                    page, d, bt.num)
    assert rc == 0 and status() == 0
    vals = cache.values(codes, sf, 1.0).astype(np.float32) * np.float32(scale)
    want = np.full((5 * bt.cols, Hkv, page, d), 7.0, np.float32)
    for b in range(5):
        n = -(-lens[b] // page)
        for p in range(n):
            here = min(page, lens[b] - p * page)
            at = want[b * bt.cols + p]
            at[:] = 0
            at[:, :here] = vals[bt.table[b, p], :, :here]
    want = I.bf16_bits_to_f32(I.f32_to_bf16_bits(want))
    assert np.array_equal(dst.float().cpu().numpy(), want)


def test_unpack_device_checks():
    rng = np.random.default_rng(201)
    bt = Batch(rng, [40, 40, 40], [0] * 3, 16)
    pool, _ = pools_fp4(rng, bt.num, 1, 16, 64)
    pool &= 0x3F
    def go(table, lens):
        dst = torch.full((3 * bt.cols, 1, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        assert attn.attn_unpack_pages_fp4(pool, dst, 1.0, dev(table), dev(lens, np.int32), 3,
                                          bt.cols, 1, 16, 64, bt.num) == 0
        return status(), (dst != 7.0).any(-1).any(-1).any(-1).cpu().numpy().reshape(3, -1)
    t = bt.table.copy()
    t[1, 1] = bt.num
    st, wrote = go(t, bt.lk)
    assert st == attn.ATTN_ERR_BOUNDS
    assert wrote[0].all() and wrote[2].all() and not wrote[1, 1] and wrote[1, 0]
    for bad in (-1, bt.cols * 16 + 1):
        st, wrote = go(bt.table, np.array([40, bad, 40]))
        assert st == attn.ATTN_ERR_SEQLENS
        assert wrote[0].all() and wrote[2].all() and not wrote[1].any()


# ------------------------------------------------------------------ decode over 4 bits

class Decode:
    """A 4-bit decode problem: finite random codes in the contexts, arbitrary bytes (NaN scales
    among them) everywhere else."""

    def __init__(self, rng, lens, Hq, Hkv, d, page, ks=0.25, vs=0.5, q_amp=1.0, N=None, spare=5,
                 num=None):
        self.lens = np.asarray(lens)
        self.bt = Batch(rng, self.lens, np.zeros(len(lens), int), page, spare=spare)
        self.Hq, self.Hkv, self.d, self.page, self.ks, self.vs = Hq, Hkv, d, page, ks, vs
        self.N = int(max(1, self.lens.max())) if N is None else N
        cols = -(-self.N // page)
        self.table = np.full((len(lens), cols), -1, np.int32)
        self.table[:, :self.bt.cols] = self.bt.table[:, :cols]
        qbits = I.f32_to_bf16_bits(rng.standard_normal((len(lens), Hq, 1, d)).astype(np.float32)
                                   * np.float32(q_amp))
        self.qv = I.bf16_bits_to_f32(qbits).astype(np.float64)[:, :, 0]
        self.q = bf16_tensor(qbits, "cuda")
        self.scale = I.default_scale(d)
        self.pools = []
        for _ in range(2):
            raw = rng.integers(0, 256, (self.bt.num, Hkv, page * (d // 2 + d // 16)),
                               dtype=np.uint8)
            cut = page * d // 2
            sf = np.full((self.bt.num, Hkv, page, d // 16), 0x7F, np.uint8)
            # scales around 1/8: 2^-4 to 2^-2
            good = rng.integers(0x18, 0x28, sf.shape, dtype=np.uint8)
            for b in range(len(lens)):
                f, s = cache.slots(np.arange(lens[b]), self.bt.table[b], page)
                sf[f, :, s] = good[f, :, s]
            raw[:, :, cut:] = sf.reshape(self.bt.num, Hkv, -1)
            self.pools.append(raw)
        self.k, self.v = (dev(p) for p in self.pools)
        self.cu = dev(np.concatenate([[0], np.cumsum(self.lens)]), np.int32)
        self.d_table = dev(self.table)
        self.alloc()

    def alloc(self):
        self.o = torch.full((len(self.lens), self.Hq, 1, self.d), float("nan"),
                            dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((len(self.lens), self.Hq), float("nan"), device="cuda")
        n = attn.attn_workspace_bytes_fp4(len(self.lens), self.Hq, self.Hkv, self.N, self.d)
        self.ws = torch.full((max(n, 16),), 0xAB, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        rc = attn.attn_fwd_paged_decode_fp4(self.q, self.k, self.v, self.o, self.lse,
                                            len(self.lens), self.Hq, self.Hkv, self.N, self.d,
                                            self.scale, self.ks, self.vs, self.cu, self.d_table,
                                            self.page, self.bt.num, self.ws, stream)
        assert rc == 0, attn.last_error()

    def context(self, which, b):
        pool, scale = self.pools[which], (self.ks, self.vs)[which]
        n = -(-self.lens[b] // self.page)
        pages = pool[self.table[b, :n]]
        codes, sf = cache.split_block(pages, self.page, self.d)
        return cache.context(cache.values(codes, sf, scale), np.arange(n), self.lens[b], self.page)

    def check(self, skip=()):
        o, lse = f64(self.o)[:, :, 0], self.lse.cpu().numpy().astype(np.float64)
        for b in range(len(self.lens)):
            if b in skip:
                continue
            if self.lens[b] == 0:
                assert not o[b].any() and np.all(lse[b] == -np.inf)
                continue
            want, wl, wa, big = cache.decode(self.qv[b], self.context(0, b), self.context(1, b),
                                             self.scale)
            vmax = np.abs(self.context(1, b)).max()
            e = 2.0 ** -18 * big
            tol = (BF16_HALF * np.abs(want) + (2.0 ** -11 + np.expm1(2 * e))[:, None] * wa
                   + 2.0 ** -18 * vmax)
            err = np.abs(o[b] - want)
            assert np.all(err <= tol), (b, float((err - tol).max()), float(err.max()))
            tl = e + 2.0 ** -17 + 2.0 ** -22 * np.abs(wl)
            assert np.all(np.abs(lse[b] - wl) <= tl), (b, float(np.abs(lse[b] - wl).max()))


EDGE_LENS = [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 7, 8, 9, 12, 16])
def test_decode_fp4(page, d, group):
    rng = np.random.default_rng(1000 + page + d + group)
    Hkv = 1 + group % 3
    w = Decode(rng, EDGE_LENS, group * Hkv, Hkv, d, page)
    w.run()
    assert status() == 0
    w.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 16])
def test_decode_fp4_splits(d, group):
    """Contexts over one, two and many splits, in a batch with as many groups as SMs (long
    splits) and in small ones (short splits)."""
    rng = np.random.default_rng(2000 + d + group)
    for lens, Hkv, page in (([511, 512, 513, 4097, 1], 2, 16), ([9000], 1, 64),
                            (list(rng.integers(1, 2500, 40)) + [2048, 2049, 0, 5000], 4, 32)):
        w = Decode(rng, lens, group * Hkv, Hkv, d, page)
        w.run()
        assert status() == 0
        w.check()
        first = w.o.clone(), w.lse.clone()
        w.run()
        torch.cuda.synchronize()
        assert torch.equal(first[0].view(torch.int16), w.o.view(torch.int16))
        assert torch.equal(first[1], w.lse)


@pytest.mark.parametrize("B,most,d,Hkv", [(333, 200, 64, 1), (97, 700, 128, 2), (33, 130, 128, 3),
                                          (32, 128, 64, 1), (700, 3, 128, 1)])
def test_decode_fp4_many_sequences(B, most, d, Hkv):
    """More sequences than a warp has lanes, empty ones among them: how the blocks are shared out,
    contexts of one block, shares that end between a context's start and its first block."""
    rng = np.random.default_rng(3000 + B)
    w = Decode(rng, rng.integers(0, most + 1, B), 2 * Hkv, Hkv, d, 16)
    w.run()
    assert status() == 0
    w.check()


def many(rng, Hkv, most, *some):
    """Lengths of enough sequences that contexts outnumber the CTAs of any variant (three an SM),
    `some` among them, in random order."""
    B = 3 * torch.cuda.get_device_properties(0).multi_processor_count // Hkv + 40
    lens = np.concatenate([rng.integers(0, most + 1, B), some]).astype(int)
    rng.shuffle(lens)
    return lens


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 7, 16])
def test_decode_fp4_many_contexts(page, d, group):
    """More contexts than CTAs, so that warps take them by themselves: odd lengths, empty ones,
    one over many warps; the same bits again on the second run."""
    rng = np.random.default_rng(3200 + page + d + group)
    lens = many(rng, 3, 200, *EDGE_LENS, 700, 1025, 5000)
    w = Decode(rng, lens, 3 * group, 3, d, page)
    w.run()
    assert status() == 0
    w.check()
    first = w.o.clone(), w.lse.clone()
    w.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0].view(torch.int16), w.o.view(torch.int16))
    assert torch.equal(first[1], w.lse)


@pytest.mark.parametrize("lens", [[0] * 700, [0] * 699 + [1], [1] * 700, [0] * 350 + [900] + [0] * 350,
                                  [128] * 600, [129] * 500])
def test_decode_fp4_many_contexts_few_tokens(lens):
    """Fewer blocks than warps, down to none."""
    rng = np.random.default_rng(3300)
    w = Decode(rng, lens, 2, 1, 128, 16)
    w.run()
    assert status() == 0
    w.check()


def test_decode_fp4_many_contexts_device_checks():
    """A NaN query, a page outside the pool, bad lengths among many contexts: each hurts its own
    rows only."""
    rng = np.random.default_rng(3400)
    lens = many(rng, 2, 300)
    lens[:8] = [200, 90, 77, 1, 128, 250, 40, 300]
    w = Decode(rng, lens, 8, 2, 128, 32, N=300)
    w.table[1, 2] = w.bt.num  # the third page of sequence 1: reads as zeros
    w.d_table = dev(w.table)
    w.q[3, 5, 0, 3] = float("nan")
    w.run()
    assert status() == attn.ATTN_ERR_BOUNDS
    assert np.isnan(w.lse[3, 5].item()) and torch.isnan(w.o[3, 5]).all()
    assert not torch.isnan(w.lse[3, :5]).any()
    w.check(skip=(1, 3))
    cu = w.cu.cpu().numpy().copy()
    w.alloc()
    cu[10] = cu[11] + 5  # sequence 10: negative; sequence 9 too long or as it is
    w.cu = dev(cu, np.int32)
    w.run()
    assert status() in (attn.ATTN_ERR_SEQLENS, attn.ATTN_ERR_BOUNDS)
    assert not f64(w.o)[10].any() and torch.all(w.lse[10] == -np.inf)
    w.check(skip=(1, 3, 9, 10))


def test_decode_fp4_all_empty():
    rng = np.random.default_rng(3100)
    w = Decode(rng, [0, 0, 0], 4, 2, 128, 16)
    w.run()
    assert status() == 0
    w.check()


def test_decode_fp4_overlaps_are_refused_and_neighbours_are_not():
    """Outputs into queries, one another or the workspace are refused and nothing is written;
    tensors that end where the next begins, as in one arena, are served."""
    rng = np.random.default_rng(3500)
    w = Decode(rng, [300, 0, 77], 8, 2, 128, 64)
    q, n = w.q, w.q.numel() * 2  # bytes, a multiple of 16; lse: 3 x 8 floats
    arena = torch.full((n + n + 96 + w.ws.numel(),), 0x5A, dtype=torch.uint8, device="cuda")

    def rows(at):
        return arena[at:at + n].view(torch.bfloat16).view(q.shape)

    def lse(at):
        return arena[at:at + 96].view(torch.float32).view(3, 8)

    ws = arena[2 * n + 96:]
    w.q, w.o, w.lse, w.ws = rows(0), rows(n), lse(2 * n), ws
    w.q.copy_(q)
    w.run()
    assert status() == 0
    w.check()
    assert torch.equal(w.q, q)
    was = arena.clone()
    for bad in (dict(o=rows(0)), dict(o=rows(n - 16)), dict(lse=lse(0)), dict(lse=lse(2 * n - 16)),
                dict(o=rows(2 * n)), dict(lse=lse(2 * n + 16)), dict(ws=arena[2 * n + 80:])):
        a = dict(o=w.o, lse=w.lse, ws=ws) | bad
        rc = attn.attn_fwd_paged_decode_fp4(w.q, w.k, w.v, a["o"], a["lse"], 3, 8, 2, w.N, 128,
                                            w.scale, w.ks, w.vs, w.cu, w.d_table, 64, w.bt.num,
                                            a["ws"])
        assert rc == attn.ATTN_ERR_INVALID and "overlap" in attn.last_error()
    assert status() == 0 and torch.equal(arena, was)


@pytest.mark.parametrize("lens", [[5000], [16384], [900, 3000]])
@pytest.mark.parametrize("d,group", [(64, 4), (64, 16), (128, 4), (128, 16)])
def test_decode_fp4_padding_changes_nothing(lens, d, group):
    """Sequences without tokens take no share of the work: a padded batch gives its live rows the
    bits that they have alone."""
    rng = np.random.default_rng(3600 + d + group)
    at = [20 + 9 * i for i in range(len(lens))]
    padded = np.zeros(50, int)
    padded[at] = lens
    w = Decode(rng, padded, 2 * group, 2, d, 64)
    w.run()
    assert status() == 0
    w.check()
    alone = Decode(rng, lens, 2 * group, 2, d, 64)
    alone.q, alone.k, alone.v = w.q[at].contiguous(), w.k, w.v
    alone.d_table, alone.bt.num = w.d_table[at].contiguous(), w.bt.num
    alone.run()
    assert status() == 0
    assert torch.equal(alone.o.view(torch.int16), w.o[at].view(torch.int16))
    assert torch.equal(alone.lse, w.lse[at])


@pytest.mark.parametrize("d", [64, 128])
def test_decode_fp4_padded_many_contexts_are_joined_in_few_parts(d):
    """Warps as workers, all but two of the batch's contexts empty: neither is cut into more than
    64 parts of an even share (65 with their ends), as what each warp leaves word of, the last
    region of the workspace, shows."""
    rng = np.random.default_rng(3700 + d)
    w = Decode(rng, [0] * 300 + [16000] + [0] * 300, 8, 2, d, 64)
    w.run()
    assert status() == 0
    w.check()
    workers = 4 * 3 * torch.cuda.get_device_properties(0).multi_processor_count
    left = w.ws[-(-workers * 16 // 256) * -256:].view(torch.int32).view(-1, 4)[:workers].cpu()
    assert sorted(left[:, 0][left[:, 2] > 0].tolist()) == [600, 601]
    assert 2 <= left[:, 2].max() <= 65


@pytest.mark.parametrize("B,Hq,Hkv,d", [(3, 4, 2, 128), (700, 2, 1, 64), (40, 64, 4, 128),
                                        (200, 32, 8, 64)])
def test_decode_fp4_without_keys(B, Hq, Hkv, d):
    """N = 0: every sequence of the batch is empty, and its rows are written all the same, eagerly
    and in a replayed graph, without pools, table or workspace; a length that is not 0 is
    reported."""
    assert attn.attn_workspace_bytes_fp4(B, Hq, Hkv, 0, d) == 0
    o = torch.full((B, Hq, 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq), float("nan"), device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")

    def run():
        rc = attn.attn_fwd_paged_decode_fp4(None, None, None, o, lse, B, Hq, Hkv, 0, d, 0.1, 1.0,
                                            1.0, cu, None, 16, 0)
        assert rc == 0, attn.last_error()

    def check():
        assert not o.view(torch.int16).any() and (lse == -np.inf).all()

    run()
    assert status() == 0
    check()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run()
    o.fill_(float("nan")), lse.fill_(float("nan"))
    g.replay()
    assert status() == 0
    check()
    cu[B] = 5
    o.fill_(float("nan")), lse.fill_(float("nan"))
    run()
    assert status() == attn.ATTN_ERR_SEQLENS
    check()


def test_decode_fp4_without_keys_takes_the_tensors_of_a_batch():
    """The same with the tensors that a serving loop passes anyway: neither q nor the workspace is
    touched."""
    rng = np.random.default_rng(3150)
    w = Decode(rng, [0] * 500, 4, 2, 128, 16)
    q, ws = w.q.clone(), w.ws.clone()
    w.N = 0
    w.run()
    assert status() == 0
    w.check()
    assert torch.equal(w.q, q) and torch.equal(w.ws, ws)


@pytest.mark.parametrize("q_amp,ks,vs", [(0.0, 1.0, 1.0), (2.0 ** -60, 1.0, 1.0), (2.0 ** 60, 2.0 ** -60, 1.0),
                                         (30.0, 0.25, 3e-20), (1.0, 1e-20, 1e20), (8.0, 0.25, 1.0)])
def test_decode_fp4_magnitudes(q_amp, ks, vs):
    """Queries and scales far from 1: Q is normalised by powers of two before f16."""
    rng = np.random.default_rng(17)
    w = Decode(rng, [700, 45], 6, 2, 128, 32, ks=ks, vs=vs, q_amp=q_amp)
    w.run()
    assert status() == 0
    w.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,B", [(1, 2), (12, 2), (4, 240)])
def test_decode_fp4_small_query_channels(d, group, B):
    """Scores that come from channels 2^16 below their head's largest, where f16 is not exact: a
    channel is off by at most 2^-25 of the largest one's power of two, a score by that times
    scale * sum |k|. (Dropped, they would leave all weights alike.)"""
    rng = np.random.default_rng(23 + d + group)
    lens = rng.integers(1, 90, B)
    lens[:2] = 700, 45
    Hkv, page = 2, 32
    w = Decode(rng, lens, group * Hkv, Hkv, d, page, ks=512.0)
    q = np.array(w.qv, np.float32) * np.float32(2.0 ** -6)
    q[:, :, 5] = 2.0 ** 10
    bits = I.f32_to_bf16_bits(q)
    w.q = bf16_tensor(bits[:, :, None], "cuda")
    w.qv = I.bf16_bits_to_f32(bits).astype(np.float64)
    codes, sf = (a.copy() for a in cache.split_block(w.pools[0], page, d))
    codes[..., 2] &= 0x0F  # channel 5 of every key: zero
    w.pools[0] = np.concatenate([codes.reshape(w.bt.num, Hkv, -1), sf.reshape(w.bt.num, Hkv, -1)], 2)
    w.k = dev(w.pools[0])
    w.run()
    assert status() == 0
    o, lse = f64(w.o)[:, :, 0], w.lse.cpu().numpy().astype(np.float64)
    for b in range(B):
        k, v = w.context(0, b), w.context(1, b)
        want, wl, wa, big = cache.decode(w.qv[b], k, v, w.scale)
        off = 2.0 ** -15 * w.scale * np.abs(k).sum(-1).max(-1).repeat(group)
        e = 2.0 ** -18 * big + off
        tol = (BF16_HALF * np.abs(want) + (2.0 ** -11 + np.expm1(2 * e))[:, None] * wa
               + 2.0 ** -18 * np.abs(v).max())
        assert np.all(np.abs(o[b] - want) <= tol)
        assert np.all(np.abs(lse[b] - wl) <= e + 2.0 ** -17 + 2.0 ** -22 * np.abs(wl))


@pytest.mark.parametrize("d", [64, 128])
def test_decode_fp4_rising_scores(d):
    """Scores that grow along the context move the running max again and again; falling ones
    leave most weights at zero."""
    rng = np.random.default_rng(18)
    for rise in (True, False):
        w = Decode(rng, [1100], 4, 1, d, 64, ks=1.0)
        codes, sf = cache.split_block(w.pools[0], 64, d)
        f, s = cache.slots(np.arange(1100), w.table[0], 64)
        # key j: all codes 1.0, scale rising from 2^-6 to 2^1 in E4M3 steps; q all ones
        step = (np.arange(1100) * 56 // 1100) if rise else 56 - np.arange(1100) * 56 // 1100
        cut = 64 * d // 2
        codes, sf = codes.copy(), sf.copy()
        codes[f, :, s] = 0x22
        sf[f, :, s] = (8 + step).astype(np.uint8)[:, None, None]
        w.pools[0] = np.concatenate([codes.reshape(w.bt.num, 1, -1), sf.reshape(w.bt.num, 1, -1)], 2)
        w.k = dev(w.pools[0])
        w.qv = np.ones_like(w.qv)
        w.q = torch.ones_like(w.q)
        w.run()
        assert status() == 0
        w.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [2, 16])
def test_decode_fp4_nan_is_not_hidden(d, group):
    """A NaN query channel makes its own row NaN, a NaN key scale the rows of its kv head, a NaN
    value scale its 16 channels; contexts of one token, of one slice and of many splits."""
    rng = np.random.default_rng(21)
    lens = [1, 20, 9000, 1, 20, 9000, 1, 9000, 40]
    Hkv, page = 2, 32
    w = Decode(rng, lens, group * Hkv, Hkv, d, page)
    codes, sf = (a.copy() for a in cache.split_block(w.pools[0], page, d))
    for b, tok in ((3, 0), (4, 11), (5, 8999)):  # keys of kv head 1
        f, s = cache.slots([tok], w.table[b], page)
        sf[f, 1, s, 1] = 0x7F
    w.k = dev(np.concatenate([codes.reshape(w.bt.num, Hkv, -1), sf.reshape(w.bt.num, Hkv, -1)], 2))
    codes, sf = (a.copy() for a in cache.split_block(w.pools[1], page, d))
    for b, tok in ((6, 0), (7, 4500)):  # values of kv head 0
        f, s = cache.slots([tok], w.table[b], page)
        sf[f, 0, s, 2] = 0x7F
    w.v = dev(np.concatenate([codes.reshape(w.bt.num, Hkv, -1), sf.reshape(w.bt.num, Hkv, -1)], 2))
    q = w.q.clone()
    q[:3, 1, 0, 17] = float("nan")
    w.q = q
    w.run()
    assert status() == 0
    o, lse = w.o.float().cpu().numpy()[:, :, 0], w.lse.cpu().numpy()
    hurt = np.zeros(o.shape, bool)
    hurt[:3, 1] = True
    hurt[3:6, group:] = True
    assert np.array_equal(np.isnan(lse), hurt[:, :, 0])
    hurt[6:8, :group, 32:48] = True
    assert np.array_equal(np.isnan(o), hurt)
    # The rest is right, as all of it is without them.
    first = w.o.clone(), w.lse.clone()
    w.q = torch.where(torch.isnan(q), torch.zeros_like(q), q)
    w.k, w.v = (dev(p) for p in w.pools)
    w.run()
    w.qv[:3, 1, 17] = 0.0
    w.check()
    # Not bit for bit: a NaN score sends its warp through the branch that moves the reference
    # max of all its heads, and a weight 2^(x - m), m not an integer, rounds to f16 by its own m.
    # The bound of check() holds for any m.
    w.o = torch.where(dev(hurt)[:, :, None], w.o, first[0])
    w.lse = torch.where(torch.isnan(first[1]), w.lse, first[1])
    w.check()


def test_decode_fp4_bad_entries():
    """A page outside the pool reads as zeros and is reported; a bad length gives O = 0 and
    LSE = -inf; the other sequences are right."""
    rng = np.random.default_rng(19)
    for page in (16, 64, 128):
        w = Decode(rng, [300, 200, 500], 4, 2, 128, page)
        bad = w.table.copy()
        bad[1, 0] = w.bt.num
        w.d_table = dev(bad)
        w.run()
        assert status() == attn.ATTN_ERR_BOUNDS
        w.check(skip=(1,))
        k, v = w.context(0, 1), w.context(1, 1)
        k[:, :page] = 0
        v[:, :page] = 0
        want, wl, wa, _ = cache.decode(w.qv[1], k, v, w.scale)
        np.testing.assert_allclose(f64(w.o)[1, :, 0], want, atol=2.0 ** -8 * np.abs(wa).max())
        np.testing.assert_allclose(w.lse[1].cpu().numpy(), wl, atol=1e-4)
    w = Decode(rng, [300, 200, 100], 4, 2, 64, 16)
    w.cu = dev(np.array([0, 300, 100, 200]), np.int32)  # sequence 1: -200 keys
    w.lens = np.array([300, 200, 100])
    w.run()
    assert status() == attn.ATTN_ERR_SEQLENS
    w.check(skip=(1,))
    assert not f64(w.o)[1].any() and torch.isinf(w.lse[1]).all()


def test_decode_fp4_table_past_the_context_is_ignored():
    rng = np.random.default_rng(20)
    w = Decode(rng, [70, 10], 4, 1, 128, 16, N=5000)
    t = w.table.copy()
    t[t < 0] = 2 ** 30
    w.d_table = dev(t)
    w.run()
    assert status() == 0
    w.check()


def test_far_pages():
    """Pools beyond 4 GB: the last page's byte offset passes 32 bits, in every entry point."""
    rng = np.random.default_rng(21)
    Hkv, d, page, num = 8, 128, 128, 60000
    bt = Batch(rng, [128], [128], page, spare=0)
    bt.table[:] = num - 1
    bt.num, bt.phys = num, np.full(128, num - 1)
    bt.d_table = dev(bt.table)
    r = Rows(rng, 128, 8, Hkv, d, 128, max_pos=128)
    kp, vp = (torch.zeros((num, Hkv, page * 72), dtype=torch.uint8, device="cuda")
              for _ in range(2))
    append_fp4(r, bt, kp, vp, 128, 0.01, 0.01)
    w = Decode(rng, [128], 8, Hkv, d, page, ks=0.01, vs=0.01)
    w.bt.num = num
    w.k, w.v = kp, vp
    w.d_table = bt.d_table
    w.run()
    dst = torch.zeros((1, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    assert attn.attn_unpack_pages_fp4(vp, dst, 0.01, bt.d_table, bt.d_lk, 1, 1, Hkv, page, d,
                                      num) == 0
    assert status() == 0
    assert not kp[0].any() and not vp[0].any()
    w.pools = [kp[num - 1:].cpu().numpy(), vp[num - 1:].cpu().numpy()]
    w.table = np.zeros((1, 1), np.int32)
    w.check()
    codes, sf = cache.quantize(r.part("v")[1].astype(np.float32), 0.01)
    want = cache.values(codes, sf, 1.0).astype(np.float32) * np.float32(0.01)
    assert np.array_equal(dst.float().cpu().numpy()[0].transpose(1, 0, 2),
                          I.bf16_bits_to_f32(I.f32_to_bf16_bits(want)))
    del kp, vp, w
    num = 20000
    bt.table[:] = num - 1
    bt.num, bt.d_table = num, dev(bt.table)
    kp, vp = (torch.zeros((num, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    append_bf16(r, bt, kp, vp, 128)
    assert status() == 0
    assert not kp[0].any() and not vp[0].any()
    assert np.array_equal(f64(vp[num - 1]).transpose(1, 0, 2), r.part("v")[1])


def test_host_tensors_are_refused():
    """Before any launch, on the current stream and on a given one, alone or among device tensors."""
    rng = np.random.default_rng(22)
    w = Decode(rng, [20], 2, 1, 128, 16)
    side = torch.cuda.Stream()
    o, lse = w.o.clone(), w.lse.clone()
    names = ("q", "k", "v", "o", "lse", "cu", "d_table", "ws")
    there = {n: getattr(w, n) for n in names}
    for some in (("q",), ("d_table",), ("o", "lse"), names):
        for n in names:
            setattr(w, n, there[n].cpu() if n in some else there[n])
        for stream in (None, 0, side, side.cuda_stream):
            with pytest.raises(attn.AttnError) as e:
                w.run(stream)
            assert e.value.code == attn.ATTN_ERR_INVALID
    for n in names:
        setattr(w, n, there[n])
    for stream in (0, side, side.cuda_stream):  # device tensors are served on each
        torch.cuda.synchronize()
        w.o.copy_(o), w.lse.copy_(lse)
        torch.cuda.synchronize()
        w.run(stream)
        assert status() == 0
        w.check()


# ------------------------------------------------------------------ a run of them together

def test_serving_run_bf16():
    """A prompt chunk appended to a bf16 cache and attended, then a decode step: norm, rotation,
    append, chunked prefill and paged decode against the oracle on the keys the pools hold."""
    rng = np.random.default_rng(30)
    Hq, Hkv, d, page = 8, 2, 128, 16
    lq = np.array([90, 33, 200])
    bt = Batch(rng, lq + 1, lq, page)  # room for one more token
    bt.lk = lq
    bt.pos = np.concatenate([np.arange(n) for n in lq])
    bt.d_lk = dev(lq, np.int32)
    r = Rows(rng, int(lq.sum()), Hq, Hkv, d, 128, max_pos=256, norm=True)
    kp, vp = (torch.zeros((bt.num, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    q = append_bf16(r, bt, kp, vp, bt.total)
    o = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    rc = attn.attn_fwd_paged_prefill(q, kp, vp, o, lse, 3, Hq, Hkv, bt.total, d,
                                     I.default_scale(d), bt.d_cu, bt.d_lk, bt.d_table, bt.cols,
                                     page, bt.num)
    assert rc == 0 and status() == 0
    bits = [t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (q, kp, vp)]
    w = I.Workload("chunk", I.MASK_PAGED_PREFILL, 3, Hq, Hkv, bt.total, d, I.default_scale(d),
                   *bits, cu_seqlens=bt.cu, block_table=bt.table, page_size=page,
                   seqlens_k=lq.astype(np.int32))
    ro, rl = oracle.attention(w)
    assert np.abs(f64(o).reshape(-1, d) - ro).max() <= 1e-2 + 2.0 ** -8 * np.abs(ro).max()
    assert np.abs(lse.cpu().numpy().reshape(-1) - rl).max() <= 1e-3
    # one token more a sequence
    st = Batch(rng, lq + 1, [1, 1, 1], page)
    st.table, st.num, st.d_table, st.cols = bt.table, bt.num, bt.d_table, bt.cols
    r2 = Rows(rng, 3, Hq, Hkv, d, 128, max_pos=256, norm=True)
    q2 = append_bf16(r2, st, kp, vp, 1)
    o2 = torch.full_like(q2, float("nan"))
    lse2 = torch.full((3, Hq), float("nan"), device="cuda")
    cu = np.concatenate([[0], np.cumsum(lq + 1)]).astype(np.int32)
    N = bt.cols * page
    ws = torch.empty(attn.attn_workspace_bytes(3, Hq, Hkv, N, d, 4, page), dtype=torch.uint8,
                     device="cuda")
    rc = attn.attn_fwd(q2, kp, vp, o2, lse2, 3, Hq, Hkv, N, d, I.default_scale(d),
                       attn.ATTN_MASK_PAGED_DECODE, 0, dev(cu), bt.d_table, page, bt.num, ws)
    assert rc == 0 and status() == 0
    bits = [t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (q2, kp, vp)]
    w = I.Workload("step", I.MASK_PAGED_DECODE, 3, Hq, Hkv, N, d, I.default_scale(d), *bits,
                   cu_seqlens=cu, block_table=bt.table, page_size=page)
    ro, rl = oracle.attention(w)
    assert np.abs(f64(o2).reshape(-1, d) - ro).max() <= 1e-2 + 2.0 ** -8 * np.abs(ro).max()
    assert np.abs(lse2.cpu().numpy().reshape(-1) - rl).max() <= 1e-3


def test_serving_run_fp4():
    """The same on a 4-bit cache: append, unpack and chunked prefill, then a captured decode step
    replayed for two tokens more, its lengths and inputs written in place."""
    rng = np.random.default_rng(31)
    Hq, Hkv, d, page = 8, 2, 128, 64
    ks, vs = 0.01, 0.01
    lq = np.array([90, 33, 200])
    bt = Batch(rng, lq + 3, lq, page)
    bt.lk = lq
    bt.pos = np.concatenate([np.arange(n) for n in lq])
    bt.d_lk = dev(lq, np.int32)
    r = Rows(rng, int(lq.sum()), Hq, Hkv, d, 128, max_pos=256, norm=True)
    kp, vp = pools_fp4(rng, bt.num, Hkv, page, d)
    q = append_fp4(r, bt, kp, vp, bt.total, ks, vs)
    kb, vb = (torch.zeros((3 * bt.cols, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    for pool, dst, s in ((kp, kb, ks), (vp, vb, vs)):
        assert attn.attn_unpack_pages_fp4(pool, dst, s, bt.d_table, bt.d_lk, 3, bt.cols, Hkv, page,
                                          d, bt.num) == 0
    o = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    flat = np.arange(3 * bt.cols, dtype=np.int32).reshape(3, -1)
    rc = attn.attn_fwd_paged_prefill(q, kb, vb, o, lse, 3, Hq, Hkv, bt.total, d,
                                     I.default_scale(d), bt.d_cu, bt.d_lk, dev(flat), bt.cols,
                                     page, 3 * bt.cols)
    assert rc == 0 and status() == 0
    bits = [t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (q, kb, vb)]
    w = I.Workload("chunk", I.MASK_PAGED_PREFILL, 3, Hq, Hkv, bt.total, d, I.default_scale(d),
                   *bits, cu_seqlens=bt.cu, block_table=flat, page_size=page,
                   seqlens_k=lq.astype(np.int32))
    ro, rl = oracle.attention(w)
    assert np.abs(f64(o).reshape(-1, d) - ro).max() <= 1e-2 + 2.0 ** -8 * np.abs(ro).max()
    assert np.abs(lse.cpu().numpy().reshape(-1) - rl).max() <= 1e-3

    # the decode step
    dw = Decode(rng, lq + 1, Hq, Hkv, d, page, ks=ks, vs=vs, N=bt.cols * page)
    dw.k, dw.v, dw.table, dw.d_table, dw.bt.num = kp, vp, bt.table, bt.d_table, bt.num
    st = Batch(rng, lq + 1, [1, 1, 1], page)
    st.table, st.num, st.d_table, st.cols = bt.table, bt.num, bt.d_table, bt.cols
    r2 = Rows(rng, 3, Hq, Hkv, d, 128, max_pos=256, norm=True)
    q2 = torch.empty((3, Hq, 1, d), dtype=torch.bfloat16, device="cuda")
    dw.q = q2

    def step():
        rc = attn.attn_append_paged_fp4(r2.part("q")[0], r2.part("k")[0], r2.part("v")[0], q2, kp,
                                        vp, ks, vs, 3, Hq, Hkv, 3, 1, d, *row_args(r2),
                                        *st.args())
        assert rc == 0, attn.last_error()
        dw.run()

    def check(lens):
        torch.cuda.synchronize()
        assert status() == 0
        dw.lens, dw.qv = lens, f64(q2)[:, :, 0]
        dw.pools = [kp.cpu().numpy(), vp.cpu().numpy()]
        dw.check()
        got = dw.context(1, 0)[:, -1]
        codes, sf = cache.quantize(r2.part("v")[1].astype(np.float32), vs)
        assert np.array_equal(got, cache.values(codes, sf, vs)[0])

    step()
    check(lq + 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for more in (2, 3):
        st.d_lk.copy_(dev(lq + more, np.int32))
        dw.cu.copy_(dev(np.concatenate([[0], np.cumsum(lq + more)]), np.int32))
        new = Rows(rng, 3, Hq, Hkv, d, 128, max_pos=256)
        r2.buf.copy_(new.buf)
        r2.x = new.x
        dw.o.fill_(float("nan"))
        g.replay()
        check(lq + more)


def test_two_graphs_share_a_workspace_and_a_stream_of_their_own():
    """Two captured decodes with one workspace, replayed one after the other on another stream
    than the one their tensors were made on."""
    rng = np.random.default_rng(32)
    a = Decode(rng, [3000, 10], 8, 2, 128, 64)
    b = Decode(rng, [1500, 2500, 700], 8, 2, 64, 16)
    b.ws = a.ws = max(a.ws, b.ws, key=lambda t: t.numel())
    a.run(), b.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for w in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            w.run(side)
        graphs.append(g)
    for w in (a, b):
        w.o.fill_(float("nan"))
    a.ws.fill_(0x5A)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            for g in graphs:
                g.replay()
    side.synchronize()
    assert attn.attn_get_status(side) == 0
    a.check()
    b.check()


def test_two_decodes_at_once():
    """Two decodes on two streams at the same time, each with its own workspace, and an append into
    a third pool beside them."""
    rng = np.random.default_rng(33)
    a = Decode(rng, list(rng.integers(500, 6000, 20)), 16, 4, 128, 64)
    b = Decode(rng, list(rng.integers(1, 4000, 9)), 32, 2, 64, 16)
    bt = Batch(rng, [400, 90], [400, 50], 16)
    r = Rows(rng, bt.total, 8, 4, 128, 128, max_pos=400, norm=True)
    _, kp, vp = pools_bf16(rng, bt, 4, 128)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        a.run(streams[0])
        b.run(streams[1])
        with torch.cuda.stream(streams[2]):
            append_bf16(r, bt, kp, vp, bt.total)
    torch.cuda.synchronize()
    assert attn.attn_get_status() == 0
    a.check()
    b.check()
    want, mag = r.want("k", bt.pos)
    close(f64(kp)[bt.phys, :, bt.slot], want, mag)


def test_many_contexts_at_once_and_replayed():
    """Two decodes of many contexts on two streams at once, each with its own workspace; then one
    captured, its lengths halved in place (some to nothing) and replayed."""
    rng = np.random.default_rng(34)
    a = Decode(rng, many(rng, 4, 300, 4000), 16, 4, 128, 128)
    b = Decode(rng, many(rng, 2, 200, 900), 32, 2, 64, 16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(streams[0])
        b.run(streams[1])
    torch.cuda.synchronize()
    assert attn.attn_get_status() == 0
    a.check()
    b.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        a.run(streams[0])
    a.lens = np.where(rng.random(len(a.lens)) < 0.2, 0, a.lens // 2)
    a.cu.copy_(dev(np.concatenate([[0], np.cumsum(a.lens)]), np.int32))
    a.o.fill_(float("nan"))
    a.ws.fill_(0x5A)
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert attn.attn_get_status() == 0
    a.check()
