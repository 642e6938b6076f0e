"""Differential attention (dense, document, chunks over pages, paged decode) and the rotation by
several axes (norm and rotation, paged append), against plain 64-bit numpy, through the C ABI.

Tolerances: oracle.diff.Rows derives those of the attention rows; of a prepared row half a step of
bf16, 2^-8 of its value, plus 2^-19 of the pair's (|a| + |b|) for the fp32 arithmetic: the norm's
sum of at most 128 squares over 8 lanes (16 fused adds and 3 shuffled ones, halved by the root), its
reciprocal root (2 ulp) and products come to less than 18 * 2^-24, a turn's three roundings to
3 * 2^-24. Outputs are pre-filled so that a row the kernels never write fails loudly."""
import numpy as np
import pytest
import torch

from oracle import cache, diff
from tiled_attention_gb300 import attn
from tiled_attention_gb300 import inputs as I
from tiled_attention_gb300.runner import bf16_tensor

pytestmark = pytest.mark.gpu

EPS = 1e-5
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2
KINDS = {"none": attn.ATTN_MASK_NONE, "causal": attn.ATTN_MASK_CAUSAL,
         "sliding": attn.ATTN_MASK_SLIDING, "sliding_bidir": attn.ATTN_MASK_SLIDING_BIDIR,
         "prefix": attn.ATTN_MASK_PREFIX_LM, "document": attn.ATTN_MASK_DOCUMENT,
         "document_bidir": attn.ATTN_MASK_DOCUMENT_BIDIR}


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


def draw(rng, *shape, amp=1.0):
    """(device bf16 tensor, its values in 64 bits)."""
    bits = I.f32_to_bf16_bits((rng.standard_normal(shape) * amp).astype(np.float32))
    return bf16_tensor(bits, "cuda"), I.bf16_bits_to_f32(bits).astype(np.float64)


def nan_like(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


class Head:
    """lam, norm weight, eps and out_scale of a layer."""

    def __init__(self, rng, Hq, d, normed=True, eps=EPS, out_scale=0.8):
        self.lam = rng.uniform(-0.5, 1.0, Hq).astype(np.float32)
        self.weight = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32) if normed else None
        self.eps, self.out_scale, self.scale = eps, out_scale, (d // 2) ** -0.5
        self.d_lam = dev(self.lam)
        self.d_weight = dev(self.weight) if normed else None

    def rows(self, q, k, v, here, step=2.0 ** -8):
        return diff.Rows(q, k, v, here, self.lam, self.scale, self.weight, self.eps, self.out_scale,
                         step)


def check(o, lse, want):
    """o [Hq, n, d], lse [Hq, 2, n] against oracle.diff.Rows."""
    err = np.abs(o - want.o)
    assert np.all(err <= want.o_tol), float(np.nanmax(err - want.o_tol))
    dead = np.isneginf(want.lse)
    assert np.array_equal(np.isneginf(lse), dead)
    err = np.abs(np.where(dead, 0, lse) - np.where(dead, 0, want.lse))
    assert np.all(err <= want.lse_tol), float(np.nanmax(err - want.lse_tol))


# ------------------------------------------------------------------ dense and document

def run_diff(h, q, k, v, kind, window=0, cu=None, B=None, stream=None):
    b, Hq, n, d = q.shape
    o, lse = nan_like(*q.shape), nan_like(b, Hq, 2, n, dtype=torch.float32)
    rc = attn.attn_fwd_diff(q, k, v, o, lse, h.d_lam, B or b, Hq, k.shape[1], n, d, h.scale, kind,
                            window, cu, h.d_weight, h.eps, h.out_scale, stream)
    assert rc == 0, attn.last_error()
    return o, lse


@pytest.mark.parametrize("mask,window", [("none", 0), ("causal", 0), ("sliding", 1),
                                         ("sliding", 100), ("sliding_bidir", 0),
                                         ("sliding_bidir", 77), ("prefix", 0), ("prefix", 150),
                                         ("prefix", 10 ** 6), ("sliding", 10 ** 6)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("normed", [False, True])
def test_dense(mask, window, d, normed):
    rng = np.random.default_rng(d + window % 1000 + normed)
    for B, Hq, Hkv, n in ((1, 1, 1, 1), (2, 3, 1, 2), (1, 2, 2, 127), (2, 4, 2, 128), (1, 4, 1, 129),
                          (3, 6, 3, 300), (1, 2, 1, 641)):
        h = Head(rng, Hq, d, normed)
        (q, qv), (k, kv), (v, vv) = (draw(rng, B, x, n, d) for x in (Hq, Hkv, Hkv))
        o, lse = run_diff(h, q, k, v, KINDS[mask], window)
        assert status() == 0
        here = diff.visible(mask, window, n)
        for b in range(B):
            check(f64(o[b]), f64(lse[b]), h.rows(qv[b], kv[b], vv[b], here))


def test_dense_many_units():
    """More work units than SMs: units follow one another in a CTA, through the ring, both Q buffers
    and every barrier's phases."""
    rng = np.random.default_rng(2)
    for d, Hq, Hkv, B, n, mask in ((128, 16, 4, 2, 1100, "causal"), (64, 32, 32, 2, 700, "causal"),
                                   (128, 64, 8, 3, 333, "none"), (64, 24, 8, 3, 1030, "sliding")):
        h = Head(rng, Hq, d)
        (q, qv), (k, kv), (v, vv) = (draw(rng, B, x, n, d) for x in (Hq, Hkv, Hkv))
        o, lse = run_diff(h, q, k, v, KINDS[mask], 300)
        assert status() == 0
        here = diff.visible(mask, 300, n)
        for b in range(B):
            check(f64(o[b]), f64(lse[b]), h.rows(qv[b], kv[b], vv[b], here))
        again, lse2 = run_diff(h, q, k, v, KINDS[mask], 300)
        assert same_bits(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("mask", ["document", "document_bidir"])
@pytest.mark.parametrize("d", [64, 128])
def test_document(mask, d):
    rng = np.random.default_rng(d)
    for lens, Hq, Hkv in (([1], 2, 1), ([5, 0, 1, 130, 0], 4, 2), ([128, 256, 127, 1, 129], 2, 2),
                          ([300, 511, 77] * 3, 16, 4)):
        n = sum(lens)
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        h = Head(rng, Hq, d)
        (q, qv), (k, kv), (v, vv) = (draw(rng, 1, x, n, d) for x in (Hq, Hkv, Hkv))
        o, lse = run_diff(h, q, k, v, KINDS[mask], 0, dev(cu), len(lens))
        assert status() == 0
        o, lse = f64(o[0]), f64(lse[0])
        for a, b in zip(cu[:-1], cu[1:]):
            cut = slice(a, b)
            if a < b:
                check(o[:, cut], lse[:, :, cut], h.rows(qv[0][:, cut], kv[0][:, cut], vv[0][:, cut],
                                                        diff.visible(mask, 0, b - a)))


@pytest.mark.parametrize("bad", [[0, 50, 40, 100], [1, 50, 60, 100], [0, 50, 60, 99], [0, 50, 60, 101]])
def test_document_bad_segments_are_reported(bad):
    rng = np.random.default_rng(4)
    h = Head(rng, 2, 128)
    q, k, v = (draw(rng, 1, 2, 100, 128)[0] for _ in range(3))
    o, _ = run_diff(h, q, k, v, attn.ATTN_MASK_DOCUMENT, 0, dev(np.array(bad, np.int32)), 3)
    assert status() == attn.ATTN_ERR_SEQLENS
    assert torch.isnan(o).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_amp,v_amp,out_scale", [(0.0, 1.0, 1.0), (20.0, 1.0, -0.5),
                                                   (1.0, 2.0 ** 100, 0.7), (1e-10, 2.0 ** -100, 2.0),
                                                   (1.0, 0.0, 1.0)])
def test_magnitudes(d, q_amp, v_amp, out_scale):
    rng = np.random.default_rng(5)
    h = Head(rng, 4, d, normed=v_amp in (0.0, 1.0), eps=1e-3, out_scale=out_scale)
    (q, qv), (k, kv), (v, vv) = (draw(rng, 1, x, 260, d, amp=a) for x, a in
                                 ((4, q_amp), (2, 1.0), (2, v_amp)))
    o, lse = run_diff(h, q, k, v, attn.ATTN_MASK_CAUSAL)
    assert status() == 0
    check(f64(o[0]), f64(lse[0]), h.rows(qv[0], kv[0], vv[0], diff.visible("causal", 0, 260)))


@pytest.mark.parametrize("d", [64, 128])
def test_rising_scores(d):
    """Scores of one map that grow along the keys move its running max again and again, the other's
    fall: the two accumulators are rescaled apart."""
    rng = np.random.default_rng(6)
    n = 700
    h = Head(rng, 2, d)
    v, vv = draw(rng, 1, 1, n, d)
    ramp = np.linspace(-60, 60, n)
    kx = np.zeros((1, 1, n, d))
    kx[..., :d // 2] = ramp[:, None] / (d // 2)
    kx[..., d // 2:] = -ramp[:, None] / (d // 2)
    kb = I.f32_to_bf16_bits(kx.astype(np.float32))
    qb = I.f32_to_bf16_bits(np.full((1, 2, n, d), 1 / h.scale, np.float32))
    kv, qv = (I.bf16_bits_to_f32(x).astype(np.float64) for x in (kb, qb))
    o, lse = run_diff(h, bf16_tensor(qb, "cuda"), bf16_tensor(kb, "cuda"), v, attn.ATTN_MASK_NONE)
    assert status() == 0
    check(f64(o[0]), f64(lse[0]), h.rows(qv[0], kv[0], vv[0], diff.visible("none", 0, n)))


def test_nan_stays_in_its_row():
    """A NaN query channel of the second map: its row's output and that map's LSE alone. Keys of NaN
    at masked places change nothing."""
    rng = np.random.default_rng(7)
    h = Head(rng, 2, 128)
    q, k, v = (draw(rng, 1, 2, 300, 128)[0] for _ in range(3))
    o, lse = run_diff(h, q, k, v, attn.ATTN_MASK_CAUSAL)
    q2, k2 = q.clone(), k.clone()
    q2[0, 1, 140, 70] = float("nan")
    k2[0, 0, 290:] = float("nan")
    o2, lse2 = run_diff(h, q2, k2, v, attn.ATTN_MASK_CAUSAL)
    assert status() == 0
    bad = torch.zeros(2, 300, dtype=torch.bool, device="cuda")
    bad[1, 140] = True
    bad[0, 290:] = True
    assert torch.equal(torch.isnan(o2[0]).all(-1), bad) and torch.equal(torch.isnan(o2[0]).any(-1), bad)
    both = torch.stack([bad, bad], 1)
    both[1, 0] = False
    assert torch.equal(torch.isnan(lse2[0]), both)
    assert same_bits(o2[0][~bad], o[0][~bad])


# ------------------------------------------------------------------ pages

class Pages:
    """Contexts of lengths lk in a shuffled pool whose other slots and pages are NaN."""

    def __init__(self, rng, lk, Hkv, d, page, amp=1.0):
        self.lk, self.page, self.Hkv, self.d = [int(x) for x in lk], page, Hkv, d
        per = [-(-x // page) for x in self.lk]
        self.num = sum(per) + 5
        self.cols = max(1, max(per))
        perm = rng.permutation(self.num)
        self.table = np.full((len(lk), self.cols), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = perm[at:at + n]
            at += n
        pools = np.full((2, self.num, Hkv, page, d), np.nan, np.float32)
        self.ctx = []
        for b, n in enumerate(self.lk):
            f, s = cache.slots(np.arange(n), self.table[b], page)
            x = (rng.standard_normal((2, n, Hkv, d)) * amp).astype(np.float32)
            x = I.bf16_bits_to_f32(I.f32_to_bf16_bits(x))
            pools[0][f, :, s], pools[1][f, :, s] = x[0], x[1]
            self.ctx.append(x.astype(np.float64).transpose(0, 2, 1, 3))
        self.k, self.v = (torch.from_numpy(p).to(torch.bfloat16).cuda() for p in pools)
        self.d_table, self.d_lk = dev(self.table), dev(np.array(self.lk, np.int32))


class Chunk(Pages):
    def __init__(self, rng, lk, lq, Hq, Hkv, d, page, normed=True):
        super().__init__(rng, lk, Hkv, d, page)
        self.lq, self.Hq = list(lq), Hq
        self.total = sum(lq)
        self.cu = dev(np.concatenate([[0], np.cumsum(lq)]).astype(np.int32))
        self.h = Head(rng, Hq, d, normed)
        self.q, self.qv = draw(rng, 1, Hq, self.total, d)

    def run(self, stream=None, **kw):
        o = nan_like(*self.q.shape)
        lse = nan_like(1, self.Hq, 2, self.total, dtype=torch.float32)
        a = dict(q=self.q, k=self.k, v=self.v, o=o, lse=lse, lam=self.h.d_lam, B=len(self.lk),
                 Hq=self.Hq, Hkv=self.Hkv, total_q=self.total, d=self.d, scale=self.h.scale,
                 norm_weight=self.h.d_weight, eps=self.h.eps, out_scale=self.h.out_scale,
                 cu_seqlens_q=self.cu, seqlens_k=self.d_lk, block_table=self.d_table,
                 max_pages=self.cols, page_size=self.page, num_pages=self.num, stream=stream)
        a.update(kw)
        rc = attn.attn_fwd_diff_paged_prefill(**a)
        assert rc == 0, attn.last_error()
        return a["o"], a["lse"]

    def check(self, o, lse, skip=()):
        o, lse = f64(o[0]), f64(lse[0])
        t0 = 0
        for b, (L, n) in enumerate(zip(self.lk, self.lq)):
            cut = slice(t0, t0 + n)
            t0 += n
            if not n or b in skip:
                continue
            here = np.arange(L)[None] <= np.arange(L - n, L)[:, None]
            k, v = self.ctx[b]
            check(o[:, cut], lse[:, :, cut], self.h.rows(self.qv[0][:, cut], k, v, here))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks(page, d):
    rng = np.random.default_rng(page + d)
    for lk, lq, Hq, Hkv in (([1], [1], 1, 1), ([300], [300], 2, 1), ([129, 40, 513], [1, 40, 200], 4, 2),
                            ([700, 128, 0, 257, 16], [130, 128, 0, 129, 16], 6, 3),
                            ([65, 90, 33] * 8, [1, 1, 1] * 8, 16, 4)):
        c = Chunk(rng, lk, lq, Hq, Hkv, d, page, normed=len(lk) != 1)
        o, lse = c.run()
        assert status() == 0
        c.check(o, lse)


def test_chunks_many_units():
    rng = np.random.default_rng(8)
    lk = rng.integers(1, 900, 23)
    lq = np.minimum(rng.integers(0, 400, 23), lk)
    for d, page, Hq, Hkv in ((128, 16, 16, 4), (64, 64, 32, 4)):
        c = Chunk(rng, lk, [int(x) for x in lq], Hq, Hkv, d, page)
        o, lse = c.run()
        assert status() == 0
        c.check(o, lse)
        o2, lse2 = c.run()
        assert same_bits(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("page", [16, 64])
def test_chunk_bad_entries(page):
    """A table entry outside the pool is reported and read as zeros; other sequences are right."""
    rng = np.random.default_rng(9)
    c = Chunk(rng, [200, 300], [200, 100], 2, 1, 128, page)
    for entry in (c.num, -1, 2 ** 31 - 1):
        table = c.table.copy()
        table[1, 1] = entry
        o, lse = c.run(block_table=dev(table))
        assert status() == attn.ATTN_ERR_BOUNDS
        c.check(o, lse, skip=(1,))
        c.ctx[1][:, :, page:2 * page] = 0
        c.check(o, lse)


@pytest.mark.parametrize("cu,lk", [([0, 50, 40], [60, 60]), ([0, 50, 101], [60, 60]),
                                   ([1, 50, 100], [60, 60]), ([0, 50, 100], [49, 60]),
                                   ([0, 50, 100], [60, 2 ** 20])])
def test_chunk_bad_lengths_are_reported(cu, lk):
    rng = np.random.default_rng(10)
    c = Chunk(rng, [60, 60], [50, 50], 2, 1, 128, 16)
    o, lse = c.run(cu_seqlens_q=dev(np.array(cu, np.int32)), seqlens_k=dev(np.array(lk, np.int32)))
    assert status() == attn.ATTN_ERR_SEQLENS
    assert torch.isnan(o).all() and torch.isnan(lse).all()


# ------------------------------------------------------------------ decode

class Decode(Pages):
    def __init__(self, rng, lk, Hq, Hkv, d, page, normed=True, amp=1.0):
        super().__init__(rng, lk, Hkv, d, page, amp)
        self.Hq = Hq
        self.h = Head(rng, Hq, d, normed)
        self.q, self.qv = draw(rng, len(lk), Hq, 1, d)
        self.N = max(1, max(self.lk))
        self.cu = dev(np.concatenate([[0], np.cumsum(self.lk)]).astype(np.int32))
        n = attn.attn_workspace_bytes_diff(len(lk), Hq, Hkv, self.N, d)
        self.ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")
        self.o = nan_like(len(lk), Hq, 1, d)
        self.lse = nan_like(len(lk), Hq, 2, dtype=torch.float32)

    def run(self, stream=None, **kw):
        a = dict(q=self.q, k=self.k, v=self.v, o=self.o, lse=self.lse, lam=self.h.d_lam,
                 B=len(self.lk), Hq=self.Hq, Hkv=self.Hkv, N=self.N, d=self.d, scale=self.h.scale,
                 norm_weight=self.h.d_weight, eps=self.h.eps, out_scale=self.h.out_scale,
                 cu_seqlens=self.cu, block_table=self.d_table, page_size=self.page,
                 num_pages=self.num, workspace=self.ws, stream=stream)
        a.update(kw)
        rc = attn.attn_fwd_diff_paged_decode(**a)
        assert rc == 0, attn.last_error()

    def check(self, skip=()):
        o, lse = f64(self.o), f64(self.lse)
        for b, n in enumerate(self.lk):
            if b in skip:
                continue
            k, v = self.ctx[b]
            # Weights as two bf16 terms, each half a step of what it rounds: 2^-8 of 2^-8.
            want = self.h.rows(self.qv[b], k, v, np.ones((1, n), bool), 2.0 ** -16)
            check(o[b], lse[b][:, :, None], want)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 7, 8, 9, 12, 16])
def test_decode(page, d, group):
    rng = np.random.default_rng(page + d + group)
    w = Decode(rng, [1, 0, 2, 15, 16, 17, 63, 64, 65, 129, 700], 2 * group, 2, d, page,
               normed=group != 2)
    w.run()
    assert status() == 0
    w.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 16])
def test_decode_splits(d, group):
    """Contexts that many workers share, and a worker's range over several contexts."""
    rng = np.random.default_rng(d + group)
    for lk in ([20000], [3000, 1, 12000, 0, 64], [5000] * 5):
        w = Decode(rng, lk, group * 2, 2, d, 64)
        w.run()
        assert status() == 0
        w.check()
        o, lse = w.o.clone(), w.lse.clone()
        for _ in range(5):
            w.run()
        assert same_bits(w.o, o) and torch.equal(w.lse, lse)


@pytest.mark.parametrize("B,most,d,Hkv,group", [(333, 200, 64, 1, 4), (97, 700, 128, 2, 2),
                                                (700, 60, 64, 2, 9), (40, 3000, 128, 8, 1)])
def test_decode_many_sequences(B, most, d, Hkv, group):
    rng = np.random.default_rng(B)
    lk = rng.integers(0, most + 1, B)
    lk[rng.integers(0, B, B // 5)] = 0
    w = Decode(rng, lk, group * Hkv, Hkv, d, 16)
    w.run()
    assert status() == 0
    w.check()


@pytest.mark.parametrize("lens", [[0], [0] * 700, [0] * 699 + [1], [0] * 350 + [900] + [0] * 350])
def test_decode_padded_batches(lens):
    rng = np.random.default_rng(11)
    w = Decode(rng, lens, 4, 2, 128, 32)
    w.run()
    assert status() == 0
    w.check()


@pytest.mark.parametrize("B,Hq,Hkv,d", [(3, 4, 2, 128), (700, 2, 1, 64), (40, 64, 4, 128)])
def test_decode_without_keys(B, Hq, Hkv, d):
    """N = 0: every row is zero and -inf; a length that is not 0 is reported."""
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    o, lse = nan_like(B, Hq, 1, d), nan_like(B, Hq, 2, dtype=torch.float32)

    def run():
        attn.check(attn.attn_fwd_diff_paged_decode(None, None, None, o, lse, None, B, Hq, Hkv, 0, d,
                                                   0.1, None, 0.0, 1.0, cu, None, 64, 0))
    run()
    assert status() == 0
    assert (o == 0).all() and (lse == float("-inf")).all()
    cu[-1] = 5
    run()
    assert status() == attn.ATTN_ERR_SEQLENS


def test_decode_bad_entries_and_lengths():
    rng = np.random.default_rng(12)
    w = Decode(rng, [300, 200, 0, 150], 4, 2, 128, 64)
    table = w.table.copy()
    table[1, 1] = w.num
    w.run(block_table=dev(table))
    assert status() == attn.ATTN_ERR_BOUNDS
    w.check(skip=(1,))
    w.ctx[1][:, :, 64:128] = 0
    w.check()
    # a length past N: that sequence is empty, the others are right (the lengths before are kept)
    w.lse.fill_(float("nan"))
    w.run(N=250, block_table=w.d_table[:, :4].contiguous())
    assert status() == attn.ATTN_ERR_SEQLENS
    w.check(skip=(0, 1))
    assert (w.o[0] == 0).all() and (w.lse[0] == float("-inf")).all()


def test_decode_nan_is_not_hidden():
    rng = np.random.default_rng(13)
    w = Decode(rng, [1, 20, 9000, 40], 4, 2, 128, 32)
    w.q[:3, 1, 0, 100] = float("nan")
    w.run()
    assert status() == 0
    bad = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    bad[:3, 1] = True
    assert torch.equal(torch.isnan(w.o[:, :, 0]).all(-1), bad)
    assert torch.equal(torch.isnan(w.lse[..., 1]), bad) and not torch.isnan(w.lse[..., 0]).any()


def test_decode_rising_scores():
    rng = np.random.default_rng(14)
    for d, group in ((64, 16), (128, 4)):
        w = Decode(rng, [1500], group, 1, d, 64)
        ramp = np.linspace(-50, 50, 1500).astype(np.float32)
        x = np.repeat(ramp[:, None, None], d, 2) / (d // 2)
        x[..., d // 2:] *= -1
        bits = I.f32_to_bf16_bits(x)
        f, s = cache.slots(np.arange(1500), w.table[0], 64)
        w.k[dev(f).long(), :, dev(s).long()] = bf16_tensor(bits, "cuda")
        w.ctx[0][0] = I.bf16_bits_to_f32(bits).astype(np.float64).transpose(1, 0, 2)
        w.q.fill_(1 / w.h.scale)
        w.qv = f64(w.q)
        w.run()
        assert status() == 0
        w.check()


# ------------------------------------------------------------------ norm and rotation

def table_of(rng, max_pos, rot):
    ang = rng.uniform(-np.pi, np.pi, (max_pos, rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


class Proj:
    """A projection's token rows (q | k | v) and how they are normed and turned."""

    def __init__(self, rng, total, Hq, Hkv, d, maps, rot, axes, order, interleaved=False, norm=False,
                 pad=0, max_pos=50):
        self.total, self.Hq, self.Hkv, self.d, self.maps = total, Hq, Hkv, d, maps
        self.rot, self.axes, self.interleaved, self.max_pos = rot, axes, interleaved, max_pos
        self.width = (Hq + 2 * Hkv) * d + pad
        self.buf, self.x = draw(rng, total, self.width)
        self.cs = table_of(rng, max_pos, max(rot, 2))
        half = rot // 2
        self.pair_axis = {"runs": [i * axes // max(1, half) for i in range(half)],
                          "turns": [i % axes for i in range(half)],
                          "any": [int(a) for a in rng.integers(0, axes, half)]}[order]
        self.pos = rng.integers(0, max_pos, (axes, total)).astype(np.int32)
        w = (1 + 0.3 * rng.standard_normal((2, d // maps))).astype(np.float32)
        self.w = [w[0], w[1]] if norm else [None, None]
        self.weights = [None if a is None else dev(a) for a in self.w]
        self.d_pos = dev(self.pos)
        self.cos_sin = dev(self.cs) if rot else None

    def part(self, name):
        lo = {"q": 0, "k": self.Hq, "v": self.Hq + self.Hkv}[name]
        h = self.Hq if name == "q" else self.Hkv
        sl = slice(lo * self.d, (lo + h) * self.d)
        return self.buf[:, sl], self.x[:, sl].reshape(-1, h, self.d)

    def want(self, name):
        return diff.prepare(self.part(name)[1], self.maps, self.w[0 if name == "q" else 1], EPS,
                            self.cs, self.pos, self.pair_axis, self.rot, self.interleaved)

    def turn(self):
        return (self.weights[0], self.weights[1], EPS, self.cos_sin, self.max_pos if self.rot else 0,
                self.rot, self.interleaved, self.axes, self.pair_axis, self.d_pos)

    def norm_rope(self, N, q=True, k=True):
        qo = nan_like(self.total // N, self.Hq, N, self.d)
        ko = nan_like(self.total // N, self.Hkv, N, self.d)
        rc = attn.attn_norm_rope_axes(self.part("q")[0] if q else None,
                                      self.part("k")[0] if k else None, qo if q else None,
                                      ko if k else None, self.total, N, self.Hq, self.Hkv, self.d,
                                      self.maps, self.width, self.width, *self.turn())
        assert rc == 0, attn.last_error()
        return qo, ko


def close(got, want, mag):
    err = np.abs(got - want)
    tol = BF16_HALF * np.abs(want) + 2.0 ** -19 * mag
    assert np.all(err <= tol), float(np.max(err - tol))


def head_major(x, N):
    t, h, d = x.shape
    return x.reshape(t // N, N, h, d).transpose(0, 2, 1, 3)


@pytest.mark.parametrize("d,maps", [(64, 1), (128, 1), (64, 2), (128, 2)])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("order", ["runs", "turns", "any"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_axes(d, maps, axes, order, interleaved):
    rng = np.random.default_rng(d + 7 * maps + 11 * axes + interleaved)
    row = d // maps
    for rot in sorted({0, 16, row // 2, row}):
        for total, N, Hq, Hkv, pad, norm in ((1, 1, 1, 1, 0, True), (6, 3, 5, 3, 8, False),
                                             (61, 61, 9, 2, 24, True)):
            r = Proj(rng, total, Hq, Hkv, d, maps, rot, axes, order, interleaved, norm, pad)
            qo, ko = r.norm_rope(N)
            assert status() == 0
            for name, got in (("q", qo), ("k", ko)):
                want, mag = r.want(name)
                close(f64(got), head_major(want, N), head_major(mag, N))


@pytest.mark.parametrize("interleaved", [False, True])
def test_one_axis_and_row_give_norm_ropes_bits(interleaved):
    rng = np.random.default_rng(15)
    for total, N in ((12, 4), (4000, 4000)):
        r = Proj(rng, total, 8, 2, 128, 1, 96, 3, "any", interleaved, True)
        r.d_pos = r.d_pos[:1].expand(3, -1).contiguous()
        qo, ko = r.norm_rope(N)
        q2, k2 = nan_like(*qo.shape), nan_like(*ko.shape)
        attn.check(attn.attn_norm_rope(r.part("q")[0], r.part("k")[0], q2, k2, total, N, 8, 2, 128,
                                       r.width, r.width, r.weights[0], r.weights[1], EPS, r.cos_sin,
                                       r.max_pos, 96, interleaved, r.d_pos[0].contiguous()))
        assert status() == 0
        assert same_bits(qo, q2) and same_bits(ko, k2)


def test_norm_rope_axes_many_tokens_and_one_tensor():
    """A warp a token and several warps a token agree bit for bit; q or k alone too."""
    rng = np.random.default_rng(16)
    r = Proj(rng, 5003, 12, 3, 64, 2, 32, 3, "turns", norm=True, max_pos=900)
    qo, ko = r.norm_rope(r.total)
    want, mag = r.want("q")
    close(f64(qo), head_major(want, r.total), head_major(mag, r.total))
    assert same_bits(r.norm_rope(r.total, k=False)[0], qo)
    assert same_bits(r.norm_rope(r.total, q=False)[1], ko)
    r.total, r.buf, r.d_pos = 40, r.buf[:40], r.d_pos[:, :40].contiguous()
    q2, k2 = r.norm_rope(40)
    assert same_bits(q2[0], qo[0, :, :40]) and same_bits(k2[0], ko[0, :, :40])


def test_norm_rope_axes_bad_positions_leave_their_rows():
    rng = np.random.default_rng(17)
    r = Proj(rng, 6, 2, 1, 128, 2, 64, 3, "runs", max_pos=10)
    pos = r.pos.copy()
    pos[0, 1], pos[1, 3], pos[2, 5] = 10, -1, 2 ** 31 - 1
    r.d_pos, r.pos = dev(pos), np.clip(pos, 0, 9)
    qo, ko = r.norm_rope(1)
    assert status() == attn.ATTN_ERR_BOUNDS
    assert torch.isnan(qo[[1, 3, 5]]).all() and torch.isnan(ko[[1, 3, 5]]).all()
    want, mag = r.want("q")
    good = [0, 2, 4]
    close(f64(qo)[good, :, 0], want[good], mag[good])


def test_norm_rope_axes_without_rotation_looks_at_no_position():
    rng = np.random.default_rng(18)
    r = Proj(rng, 6, 2, 1, 128, 2, 0, 3, "runs", norm=True)
    r.d_pos, r.pair_axis = None, None
    qo, _ = r.norm_rope(1)
    assert status() == 0
    r.pair_axis = []
    want, mag = r.want("q")
    close(f64(qo)[:, :, 0], want, mag)


# ------------------------------------------------------------------ append

def append(r, pg, lq, N, behind=0, q=True, **kw):
    qo = nan_like(r.total // N, r.Hq, N, r.d)
    cu = np.concatenate([[0], np.cumsum(lq)]).astype(np.int32)
    a = dict(cu=dev(cu), lk=pg.d_lk, table=pg.d_table)
    a.update(kw)
    rc = attn.attn_append_paged_axes(r.part("q")[0] if q else None, r.part("k")[0], r.part("v")[0],
                                     qo if q else None, pg.k, pg.v, len(lq), r.Hq, r.Hkv, r.total, N,
                                     r.d, r.maps, r.width, r.width, r.width, *r.turn(), a["cu"],
                                     a["lk"], a["table"], pg.cols, pg.page, pg.num)
    assert rc == 0, attn.last_error()
    return qo


def new_slots(pg, lq):
    phys, slot = [], []
    for b, n in enumerate(lq):
        f, s = cache.slots(np.arange(pg.lk[b] - n, pg.lk[b]), pg.table[b], pg.page)
        phys.append(f), slot.append(s)
    return np.concatenate(phys).astype(int), np.concatenate(slot).astype(int)


RAGGED = [([1], [1], 0), ([40, 7, 0, 129, 16], [3, 7, 0, 1, 16], 3), ([65, 64, 63, 128], [1, 1, 1, 1], 0),
          ([300, 1, 48], [210, 1, 33], 2)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,maps,rot,axes,order,interleaved,norm", [
    (64, 1, 64, 3, "runs", False, True), (64, 2, 32, 3, "turns", False, False),
    (128, 1, 48, 2, "any", True, True), (128, 2, 64, 4, "runs", False, True),
    (128, 2, 0, 1, "runs", False, False)])
def test_append_axes(page, d, maps, rot, axes, order, interleaved, norm):
    rng = np.random.default_rng(page + d + rot)
    for (lk, lq, behind), (Hq, Hkv) in zip(RAGGED, ((4, 4), (6, 2), (8, 1), (5, 5))):
        pg = Pages(rng, lk, Hkv, d, page)
        real = sum(lq)
        r = Proj(rng, real + behind, Hq, Hkv, d, maps, rot, axes, order, interleaved, norm)
        if rot and behind:  # positions of rows behind the last sequence are not looked at
            r.d_pos[:, real:] = -5
        N = 1 if max(lq) == 1 else r.total
        was = [p.clone() for p in (pg.k, pg.v)]
        qo = append(r, pg, lq, N)
        assert status() == 0
        want, mag = r.want("q")
        tok = f64(qo).transpose(0, 2, 1, 3).reshape(r.total, Hq, d)
        close(tok[:real], want[:real], mag[:real])
        assert np.isnan(tok[real:]).all(), "rows behind the last sequence were written"
        phys, slot = new_slots(pg, lq)
        want, mag = r.want("k")
        close(f64(pg.k)[phys, :, slot], want[:real], mag[:real])
        assert np.array_equal(f64(pg.v)[phys, :, slot], r.part("v")[1][:real])
        f, s = torch.from_numpy(phys), torch.from_numpy(slot)
        for got, old in zip((pg.k, pg.v), was):  # every other slot as it was
            got[f, :, s] = old[f, :, s]
            assert same_bits(got, old)


def test_append_axes_without_queries_and_one_axis():
    rng = np.random.default_rng(19)
    pg = Pages(rng, [50, 20], 2, 128, 16)
    r = Proj(rng, 31, 4, 2, 128, 1, 128, 2, "turns", norm=True, max_pos=64)
    at = np.concatenate([np.arange(20, 50), [19]]).astype(np.int32)
    r.d_pos = dev(np.stack([at, at]))
    ref = [p.clone() for p in (pg.k, pg.v)]
    append(r, pg, [30, 1], r.total, q=False)
    cu = dev(np.array([0, 30, 31], np.int32))
    attn.check(attn.attn_append_paged(None, r.part("k")[0], r.part("v")[0], None, ref[0], ref[1], 2, 4,
                                      2, 31, 31, 128, r.width, r.width, r.width, None, r.weights[1],
                                      EPS, r.cos_sin, 64, 128, False, cu, pg.d_lk, pg.d_table, pg.cols,
                                      16, pg.num))
    assert status() == 0
    assert same_bits(pg.k, ref[0]) and same_bits(pg.v, ref[1])


@pytest.mark.parametrize("fault", ["long", "decreasing", "past", "page", "negative page", "position"])
def test_append_axes_device_checks(fault):
    """Bad lengths, pages and positions are reported and never written through; the other tokens
    are written."""
    rng = np.random.default_rng(20)
    pg = Pages(rng, [40, 20, 33], 2, 128, 16)
    lq = [5, 2, 4]
    r = Proj(rng, 11, 2, 2, 128, 2, 64, 3, "runs")
    cu, lk, table = np.array([0, 5, 7, 11], np.int32), np.array(pg.lk, np.int32), pg.table.copy()
    code, hurt = attn.ATTN_ERR_SEQLENS, [5, 6]  # tokens whose K and V stay out
    if fault == "long":
        lk[1] = pg.cols * 16 + 1
    elif fault == "decreasing":
        cu[2] = 3  # rows 3 and 4 are of two sequences: which is found varies, no slot is checked
    elif fault == "past":
        lk[1] = 1
    elif fault in ("page", "negative page"):
        table[1, 1] = pg.num if fault == "page" else -7
        code = attn.ATTN_ERR_BOUNDS
    else:
        pos = r.pos.copy()
        pos[2, 5], pos[1, 6] = 50, -1
        r.d_pos = dev(pos)
        code = attn.ATTN_ERR_BOUNDS
    was = [p.clone() for p in (pg.k, pg.v)]
    append(r, pg, lq, r.total, cu=dev(cu), lk=dev(lk), table=dev(table))
    assert status() == code
    if fault == "decreasing":
        return
    phys, slot = new_slots(pg, lq)
    want, mag = r.want("k")
    ok = [t for t in range(11) if t not in hurt]
    close(f64(pg.k)[phys[ok], :, slot[ok]], want[ok], mag[ok])
    f, s = torch.from_numpy(phys[ok]), torch.from_numpy(slot[ok])
    for got, old in zip((pg.k, pg.v), was):
        got[f, :, s] = old[f, :, s]
        assert same_bits(got, old)


# ------------------------------------------------------------------ together

class Layer:
    """Projections of B prompts and of single tokens after them, through append_axes (two maps), chunk
    attention and decode over the cache; the rows a definition gives in 64 bits from the cache's
    own bf16 keys."""

    def __init__(self, rng, lens, steps, Hq, Hkv, d, page):
        self.lens, self.steps = lens, steps
        self.pg = Pages(rng, [n + steps for n in lens], Hkv, d, page)
        self.h = Head(rng, Hq, d)
        self.r = [Proj(rng, n + steps, Hq, Hkv, d, 2, d // 2, 3, "runs", norm=True, max_pos=400)
                  for n in lens]
        for r in self.r[1:]:
            r.w, r.weights, r.cs, r.cos_sin = (self.r[0].w, self.r[0].weights, self.r[0].cs,
                                               self.r[0].cos_sin)
        self.Hq, self.Hkv, self.d, self.page = Hq, Hkv, d, page
        self.pg.k.fill_(float("nan")), self.pg.v.fill_(float("nan"))

    def rows(self, take):
        """Token rows and positions of take(r, b), sequence after sequence."""
        buf = torch.cat([take(r.buf) for r in self.r])
        pos = torch.cat([take(r.d_pos.T) for r in self.r]).T.contiguous()
        return buf, pos

    def append(self, buf, pos, lq, lk, N):
        r, total, w = self.r[0], buf.shape[0], buf.shape[1]
        qo = nan_like(total // N, self.Hq, N, self.d)
        cu = dev(np.concatenate([[0], np.cumsum(lq)]).astype(np.int32))
        kv = self.Hkv * self.d
        q, k, v = buf[:, :w - 2 * kv], buf[:, w - 2 * kv:w - kv], buf[:, w - kv:]
        attn.check(attn.attn_append_paged_axes(
            q, k, v, qo, self.pg.k, self.pg.v, len(lq), self.Hq, self.Hkv, total, N, self.d, 2, w, w,
            w, r.weights[0], r.weights[1], EPS, r.cos_sin, 400, self.d // 2, False, 3, r.pair_axis,
            pos, cu, lk, self.pg.d_table, self.pg.cols, self.page, self.pg.num))
        return qo, cu


def test_serving_run():
    """Two chunks of every prompt, then single tokens: each output against the definition over the
    bf16 keys and values that the run itself has put into the cache, and the dense form of the whole
    against the same."""
    rng = np.random.default_rng(21)
    lens, steps, Hq, Hkv, d, page = [200, 77, 130], 3, 4, 2, 128, 16
    s = Layer(rng, lens, steps, Hq, Hkv, d, page)
    h = s.h
    done = [0] * 3
    dense = []
    for b, r in enumerate(s.r):  # the dense form: norm_rope_axes, then causal attention
        qo, ko = r.norm_rope(r.total)
        v = r.part("v")[0].reshape(r.total, Hkv, d).transpose(0, 1)[None].contiguous()
        dense.append((qo, ko, v, *run_diff(h, qo, ko, v, attn.ATTN_MASK_CAUSAL)))
    for part in range(2):
        lq = [n // 2 if part == 0 else n - n // 2 for n in lens]
        done = [a + n for a, n in zip(done, lq)]
        lk = dev(np.array(done, np.int32))
        buf = torch.cat([r.buf[e - n:e] for r, e, n in zip(s.r, done, lq)])
        pos = torch.cat([r.d_pos[:, e - n:e] for r, e, n in zip(s.r, done, lq)], 1).contiguous()
        qo, cu = s.append(buf, pos, lq, lk, buf.shape[0])
        o, lse = nan_like(*qo.shape), nan_like(1, Hq, 2, qo.shape[2], dtype=torch.float32)
        attn.check(attn.attn_fwd_diff_paged_prefill(
            qo, s.pg.k, s.pg.v, o, lse, h.d_lam, 3, Hq, Hkv, qo.shape[2], d, h.scale, h.d_weight,
            h.eps, h.out_scale, cu, lk, s.pg.d_table, s.pg.cols, page, s.pg.num))
        t0 = 0
        for b, (e, n) in enumerate(zip(done, lq)):
            dq, dk, dv, do, dl = dense[b]
            assert same_bits(qo[0, :, t0:t0 + n], dq[0, :, e - n:e])
            here = np.arange(e)[None] <= np.arange(e - n, e)[:, None]
            want = h.rows(f64(dq[0, :, e - n:e]), f64(dk[0, :, :e]), f64(dv[0, :, :e]), here)
            check(f64(o[0, :, t0:t0 + n]), f64(lse[0, :, :, t0:t0 + n]), want)
            check(f64(do[0, :, e - n:e]), f64(dl[0, :, :, e - n:e]), want)
            t0 += n
    ws = torch.empty(attn.attn_workspace_bytes_diff(3, Hq, Hkv, 256, d), dtype=torch.uint8,
                     device="cuda")
    table = torch.full((3, 256 // page), -1, dtype=torch.int32, device="cuda")
    table[:, :s.pg.cols] = s.pg.d_table
    for step in range(steps):
        done = [a + 1 for a in done]
        lk = dev(np.array(done, np.int32))
        buf = torch.cat([r.buf[e - 1:e] for r, e in zip(s.r, done)])
        pos = torch.cat([r.d_pos[:, e - 1:e] for r, e in zip(s.r, done)], 1).contiguous()
        qo, _ = s.append(buf, pos, [1] * 3, lk, 1)
        o, lse = nan_like(3, Hq, 1, d), nan_like(3, Hq, 2, dtype=torch.float32)
        cu = dev(np.concatenate([[0], np.cumsum(done)]).astype(np.int32))
        attn.check(attn.attn_fwd_diff_paged_decode(qo, s.pg.k, s.pg.v, o, lse, h.d_lam, 3, Hq, Hkv,
                                                   256, d, h.scale, h.d_weight, h.eps, h.out_scale,
                                                   cu, table, page, s.pg.num, ws))
        for b, e in enumerate(done):
            dq, dk, dv, _, _ = dense[b]
            assert same_bits(qo[b, :, 0], dq[0, :, e - 1])
            want = h.rows(f64(qo[b]), f64(dk[0, :, :e]), f64(dv[0, :, :e]), np.ones((1, e), bool))
            check(f64(o[b]), f64(lse[b])[:, :, None], want)
    assert status() == 0


def test_captured_and_replayed():
    """Append, chunk attention, decode and the dense form captured into one graph on a stream of its
    own, replayed with other inputs written in place."""
    rng = np.random.default_rng(22)
    c = Chunk(rng, [200, 90], [70, 90], 4, 2, 128, 32)
    w = Decode(rng, [500, 0, 129], 8, 2, 64, 16)
    h = Head(rng, 4, 128)
    q, k, v = (draw(rng, 1, x, 300, 128)[0] for x in (4, 2, 2))
    r = Proj(rng, 40, 4, 2, 128, 2, 64, 3, "turns")
    outs = dict(o=nan_like(*c.q.shape), lse=nan_like(1, 4, 2, c.total, dtype=torch.float32))
    d_o, d_l = nan_like(*q.shape), nan_like(1, 4, 2, 300, dtype=torch.float32)
    qo, ko = nan_like(10, 4, 4, 128), nan_like(10, 2, 4, 128)

    def all_of(stream):
        c.run(stream, **outs)
        w.run(stream)
        attn.check(attn.attn_fwd_diff(q, k, v, d_o, d_l, h.d_lam, 1, 4, 2, 300, 128, h.scale,
                                      attn.ATTN_MASK_CAUSAL, 0, None, h.d_weight, h.eps, h.out_scale,
                                      stream))
        attn.check(attn.attn_norm_rope_axes(r.part("q")[0], r.part("k")[0], qo, ko, 40, 4, 4, 2, 128, 2,
                                            r.width, r.width, *r.turn(), stream))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_of(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            all_of(side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t, name in ((c.q, "c"), (w.q, "w"), (q, "q")):
            new, vals = draw(rng, *t.shape)
            t.copy_(new)
            if name == "c":
                c.qv = vals
            elif name == "w":
                w.qv = vals
        lens = [int(x) for x in rng.integers(0, 500, 3)]  # shorter contexts in the same pages
        r.buf.copy_(draw(rng, *r.buf.shape)[0])
        r.x = f64(r.buf)
        for b, n in enumerate(lens):
            n = w.lk[b] = min(n, w.ctx[b].shape[2])
            w.ctx[b] = w.ctx[b][:, :, :n]
        w.cu.copy_(dev(np.concatenate([[0], np.cumsum(w.lk)]).astype(np.int32)))
        for t in (outs["o"], outs["lse"], w.o, w.lse, d_o, d_l, qo, ko):
            t.fill_(float("nan"))
        g.replay()
        assert status() == 0
        c.check(outs["o"], outs["lse"])
        w.check()
        want = h.rows(f64(q[0]), f64(k[0]), f64(v[0]), diff.visible("causal", 0, 300))
        check(f64(d_o[0]), f64(d_l[0]), want)
        for name, got in (("q", qo), ("k", ko)):
            x, mag = r.want(name)
            close(f64(got), head_major(x, 4), head_major(mag, 4))


def test_two_at_once_and_a_shared_workspace():
    """Decodes on two streams at once with a workspace each, and two graphs that share one, replayed
    one after the other."""
    rng = np.random.default_rng(23)
    a = Decode(rng, [9000, 300], 8, 2, 128, 64)
    b = Decode(rng, [700] * 40, 4, 4, 64, 16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(streams[0])
        b.run(streams[1])
    assert status() == 0
    a.check(), b.check()
    a.o.fill_(float("nan")), b.o.fill_(float("nan"))
    n = max(a.ws.numel(), b.ws.numel())
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs = []
    torch.cuda.synchronize()
    for w in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            w.run(streams[0], workspace=ws)
        graphs.append(g)
    with torch.cuda.stream(streams[1]):
        for _ in range(5):
            for g in graphs:
                g.replay()
    assert status() == 0
    a.check(), b.check()


@pytest.mark.parametrize("d", [64, 128])
def test_large_values_under_rising_scores(d):
    """Values of 2^70 beside weights that grow by 2^57 along a row: products stay finite."""
    rng = np.random.default_rng(25)
    n = 700
    w = Decode(rng, [n], 2, 1, d, 64, normed=False)
    h = w.h
    ramp = np.linspace(-20, 20, n)
    kx = np.zeros((n, d))
    kx[:, :d // 2], kx[:, d // 2:] = ramp[:, None] / (d // 2), -ramp[:, None] / (d // 2)
    vx = rng.standard_normal((n, d)) * 2.0 ** 70
    kb, vb = (I.f32_to_bf16_bits(x.astype(np.float32)) for x in (kx, vx))
    kv, vv = (I.bf16_bits_to_f32(x).astype(np.float64)[None] for x in (kb, vb))
    qb = I.f32_to_bf16_bits(np.full((1, 2, n, d), 1 / h.scale, np.float32))
    qv = I.bf16_bits_to_f32(qb).astype(np.float64)
    q, k, v = (bf16_tensor(x, "cuda") for x in (qb, kb[None, None], vb[None, None]))
    o, lse = run_diff(h, q, k, v, attn.ATTN_MASK_NONE)
    f, s = cache.slots(np.arange(n), w.table[0], 64)
    f, s = dev(f, np.int64), dev(s, np.int64)
    w.k[f, 0, s], w.v[f, 0, s] = k[0, 0], v[0, 0]
    w.run(q=q[:, :, -1:].contiguous())
    assert status() == 0
    want = h.rows(qv[0], kv, vv, diff.visible("none", 0, n))
    check(f64(o[0]), f64(lse[0]), want)
    want = h.rows(qv[0][:, -1:], kv, vv, np.ones((1, n), bool))
    check(f64(w.o[0]), f64(w.lse[0])[:, :, None], want)


def test_shared_pages():
    """Two sequences that hold the same pages of a common prefix."""
    rng = np.random.default_rng(26)
    c = Chunk(rng, [200, 300], [60, 90], 4, 2, 128, 32)
    w = Decode(rng, [500, 129, 700], 8, 2, 64, 16)
    for x, n in ((c, 192), (w, 128)):
        x.table[1, :n // x.page] = x.table[0, :n // x.page]
        x.d_table = dev(x.table)
        x.ctx[1][:, :, :n] = x.ctx[0][:, :, :n]
    o, lse = c.run()
    w.run()
    assert status() == 0
    c.check(o, lse), w.check()


@pytest.mark.parametrize("mask,window", [("none", 0), ("causal", 0), ("sliding", 200),
                                         ("sliding_bidir", 130), ("prefix", 300), ("document", 0),
                                         ("document_bidir", 0)])
def test_more_units_than_four_an_sm(mask, window):
    """d = 64: more than four 128-row units an SM go two CTAs an SM. A few planes of each."""
    rng = np.random.default_rng(28)
    doc = mask.startswith("document")
    B, Hq, Hkv, n, cuts = (1, 48, 12, 1900, [0, 1, 130, 130, 1299, 1900]) if doc else (
        4, 16, 4, 1399, [0, 1399])
    h = Head(rng, Hq, 64)
    (q, qv), (k, kv), (v, vv) = (draw(rng, B, x, n, 64) for x in (Hq, Hkv, Hkv))
    o, lse = run_diff(h, q, k, v, KINDS[mask], window, dev(np.array(cuts, np.int32)) if doc else None,
                      len(cuts) - 1 if doc else None)
    assert status() == 0
    lam = h.lam
    for b, hq in ((0, 0), (B - 1, Hq - 1), (B // 2, Hq // 2 + 1)):
        h.lam = lam[hq:hq + 1]
        g = hq // (Hq // Hkv)
        for lo, hi in zip(cuts, cuts[1:]):
            if lo == hi:
                continue
            want = h.rows(qv[b, hq:hq + 1, lo:hi], kv[b, g:g + 1, lo:hi], vv[b, g:g + 1, lo:hi],
                          diff.visible(mask, window, hi - lo))
            check(f64(o[b, hq:hq + 1, lo:hi]), f64(lse[b, hq:hq + 1, :, lo:hi]), want)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_more_chunk_units_than_four_an_sm(page):
    rng = np.random.default_rng(29 + page)
    c = Chunk(rng, [900, 33, 777, 640, 128], [400, 33, 129, 1, 128], 48, 3, 64, page)
    o, lse = c.run()
    assert status() == 0
    c.check(o, lse)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (12, 1), (6, 2), (32, 2), (16, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_share_a_tile(Hq, Hkv, d):
    """Chunks and document segments whose last 128-row tile has few rows, of heads that share a kv
    head: powers of two that divide the group go into one tile."""
    rng = np.random.default_rng(30 + Hq + d)
    lq = [1, 8, 9, 16, 17, 32, 33, 64, 65, 0, 130, 192, 193, 257, 5]
    c = Chunk(rng, [n + int(x) for n, x in zip(lq, rng.integers(0, 300, len(lq)))], lq, Hq, Hkv, d, 16)
    o, lse = c.run()
    assert status() == 0
    c.check(o, lse)
    n, h = sum(lq), c.h
    cu = np.concatenate([[0], np.cumsum(lq)]).astype(np.int32)
    (k, kv), (v, vv) = (draw(rng, 1, Hkv, n, d) for _ in range(2))
    for mask in ("document", "document_bidir"):
        o, lse = run_diff(h, c.q, k, v, KINDS[mask], 0, dev(cu), len(lq))
        assert status() == 0
        o, lse = f64(o[0]), f64(lse[0])
        for a, b in zip(cu[:-1], cu[1:]):
            if a < b:
                check(o[:, a:b], lse[:, :, a:b], h.rows(c.qv[0][:, a:b], kv[0][:, a:b],
                                                        vv[0][:, a:b], diff.visible(mask, 0, b - a)))


@pytest.mark.parametrize("n", [1, 7, 8, 17, 40, 64, 65, 150, 192, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_short_dense_rows_share_a_tile(n, d):
    rng = np.random.default_rng(31 + n + d)
    h = Head(rng, 24, d)
    for mask, window in (("none", 0), ("causal", 0), ("sliding", 9), ("prefix", 5)):
        (q, qv), (k, kv), (v, vv) = (draw(rng, 9, x, n, d) for x in (24, 3, 3))
        o, lse = run_diff(h, q, k, v, KINDS[mask], window)
        assert status() == 0
        for b in range(0, 9, 4):
            check(f64(o[b]), f64(lse[b]), h.rows(qv[b], kv[b], vv[b], diff.visible(mask, window, n)))


def test_prefills_at_once():
    """Dense, packed and chunk attention on three streams at once, each of more units than the GPU
    holds, give the bits that they give alone."""
    rng = np.random.default_rng(27)
    h = Head(rng, 16, 128)
    q, k, v = (draw(rng, 2, x, 1500, 128)[0] for x in (16, 4, 4))
    h64 = Head(rng, 8, 64)
    q64, k64, v64 = (draw(rng, 1, x, 5000, 64)[0] for x in (8, 4, 4))
    cu = dev(np.array([0, 1300, 1300, 3100, 5000], np.int32))
    lk = rng.integers(600, 900, 16)
    c = Chunk(rng, lk, [300] * 16, 8, 2, 128, 32)

    calls = [lambda: run_diff(h, q, k, v, attn.ATTN_MASK_CAUSAL),
             lambda: run_diff(h64, q64, k64, v64, attn.ATTN_MASK_DOCUMENT, cu=cu, B=4), c.run]
    alone = [call() for call in calls]
    assert status() == 0
    for _ in range(3):
        got = []
        for call in calls:
            with torch.cuda.stream(torch.cuda.Stream()):
                got.append(call())
        assert status() == 0
        for (o, lse), (po, pl) in zip(got, alone):
            assert same_bits(o, po) and torch.equal(lse, pl)


def test_far_pages():
    """Pools of more than 2^32 bytes: appended to, read by a chunk and by a decode at their end."""
    Hq, Hkv, d, page = 4, 2, 128, 64
    num = (5 << 30) // (Hkv * page * d * 2)
    k, v = (torch.zeros((num, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rng = np.random.default_rng(24)
    n = 150
    r = Proj(rng, n, Hq, Hkv, d, 2, 64, 3, "runs")
    table = dev(np.array([[num - 1, num - 2, num - 3]], np.int32))
    lk, cu = dev(np.array([n], np.int32)), dev(np.array([0, n], np.int32))
    qo = nan_like(1, Hq, n, d)
    h = Head(rng, Hq, d)
    attn.check(attn.attn_append_paged_axes(r.part("q")[0], r.part("k")[0], r.part("v")[0], qo, k, v, 1,
                                           Hq, Hkv, n, n, d, 2, r.width, r.width, r.width, *r.turn(),
                                           cu, lk, table, 3, page, num))
    o, lse = nan_like(1, Hq, n, d), nan_like(1, Hq, 2, n, dtype=torch.float32)
    attn.check(attn.attn_fwd_diff_paged_prefill(qo, k, v, o, lse, h.d_lam, 1, Hq, Hkv, n, d, h.scale,
                                                h.d_weight, h.eps, h.out_scale, cu, lk, table, 3, page,
                                                num))
    o1, lse1 = nan_like(1, Hq, 1, d), nan_like(1, Hq, 2, dtype=torch.float32)
    ws = torch.empty(attn.attn_workspace_bytes_diff(1, Hq, Hkv, n, d), dtype=torch.uint8, device="cuda")
    q1 = qo[:, :, -1:].contiguous()
    attn.check(attn.attn_fwd_diff_paged_decode(q1, k, v, o1, lse1, h.d_lam, 1, Hq, Hkv, n, d, h.scale,
                                               h.d_weight, h.eps, h.out_scale, cu, table, page, num,
                                               ws))
    assert status() == 0
    _, ko = r.norm_rope(n)
    vv = r.part("v")[1].transpose(1, 0, 2)
    want = h.rows(f64(qo[0]), f64(ko[0]), vv, diff.visible("causal", 0, n))
    check(f64(o[0]), f64(lse[0]), want)
    want = h.rows(f64(q1[0]), f64(ko[0]), vv, np.ones((1, n), bool))
    check(f64(o1[0]), f64(lse1[0])[:, :, None], want)
