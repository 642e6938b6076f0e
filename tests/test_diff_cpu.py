"""Differential attention's and the several-axis row entry points' argument checks (before any CUDA
call), and their oracle's own pins. CPU only."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import cache, diff
from tiled_attention_gb300 import attn, build

INVALID, UNSUPPORTED, WORKSPACE = (attn.ATTN_ERR_INVALID, attn.ATTN_ERR_UNSUPPORTED,
                                   attn.ATTN_ERR_WORKSPACE)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()
    return attn.lib()


class _Ptr:
    """Stands in for a device tensor in calls that fail validation: never dereferenced."""

    def __init__(self, addr=1 << 20, device=0, n=0):
        self.addr, self.device, self.n = addr, device, n

    def data_ptr(self):
        return self.addr

    def get_device(self):
        return self.device

    def numel(self):
        return self.n

    def element_size(self):
        return 1


T = _Ptr()
ODD = _Ptr((1 << 20) | 8)
HALF = _Ptr((1 << 20) | 2)


def _norm_rope(**kw):
    a = dict(q=T, k=T, q_out=_Ptr(1 << 24), k_out=_Ptr(1 << 25), total=8, N=4, Hq=4, Hkv=2, d=128,
             maps=2, q_stride=512, k_stride=256, q_weight=None, k_weight=None, eps=1e-6, cos_sin=T,
             max_pos=16, rot_dim=64, interleaved=False, axes=3, pair_axis=[0, 1, 2, 0] * 8,
             positions=T, stream=0)
    a.update(kw)
    return attn.attn_norm_rope_axes(**a)


def _append(**kw):
    a = dict(q=T, k=T, v=T, q_out=_Ptr(1 << 24), k_pool=_Ptr(1 << 28), v_pool=_Ptr(1 << 29), B=2,
             Hq=4, Hkv=2, total_q=8, N=8, d=128, maps=2, q_stride=512, k_stride=256, v_stride=256,
             q_weight=None, k_weight=None, eps=1e-6, cos_sin=T, max_pos=16, rot_dim=64,
             interleaved=False, axes=3, pair_axis=bytes([0, 1, 2, 0] * 8), positions=T,
             cu_seqlens_q=T, seqlens_k=T, block_table=T, max_pages=4, page_size=64, num_pages=8,
             stream=0)
    a.update(kw)
    return attn.attn_append_paged_axes(**a)


ROW_REFUSALS = [
    (dict(maps=0), INVALID),
    (dict(maps=3), INVALID),
    (dict(d=96), UNSUPPORTED),
    (dict(d=32, maps=1), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED),
    (dict(rot_dim=128, pair_axis=[0] * 64), INVALID),  # more than a map's 64 channels
    (dict(rot_dim=-16, pair_axis=None), INVALID),
    (dict(rot_dim=24, pair_axis=[0] * 12), UNSUPPORTED),
    (dict(axes=0), INVALID),
    (dict(axes=5), INVALID),
    (dict(axes=2), INVALID),  # pair_axis names a third
    (dict(pair_axis=[0] * 31 + [3]), INVALID),
    (dict(pair_axis=None), INVALID),
    (dict(positions=None), INVALID),
    (dict(max_pos=0), INVALID),
    (dict(cos_sin=None), INVALID),
    (dict(cos_sin=ODD), INVALID),
    (dict(q=ODD), INVALID),
    (dict(k=ODD), INVALID),
    (dict(q_out=None), INVALID),
    (dict(q_out=ODD), INVALID),
    (dict(q_stride=504), INVALID),  # below the heads' width
    (dict(k_stride=260), INVALID),  # rows not 16-byte aligned
    (dict(q_weight=ODD), INVALID),
    (dict(q_weight=T, eps=-1.0), INVALID),
    (dict(k_weight=T, eps=float("nan")), INVALID),
    (dict(N=3), INVALID),  # 8 tokens are not rows of 3
    (dict(N=0), INVALID),
    (dict(Hq=-1), INVALID),
    (dict(Hq=2 ** 30, q_stride=2 ** 37), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", ROW_REFUSALS + [
    (dict(k_out=None), INVALID),
    (dict(k_out=ODD), INVALID),
    (dict(total=-8), INVALID),
    (dict(k_out=_Ptr(1 << 24)), INVALID),  # q_out's place
    (dict(k_out=_Ptr((1 << 20) + 4096)), INVALID),  # inside q
    (dict(q_out=_Ptr((1 << 20) - 16)), INVALID),
    (dict(q=None, k=None), INVALID),
    (dict(positions=_Ptr((1 << 24) + 4)), INVALID),  # inside q_out
    (dict(positions=_Ptr((1 << 25) - 4)), INVALID),  # k_out
])
def test_norm_rope_axes_refusals(kw, code):
    assert _norm_rope(**kw) == code
    assert attn.last_error()


@pytest.mark.parametrize("kw,code", ROW_REFUSALS + [
    (dict(Hkv=0), INVALID),
    (dict(B=-1), INVALID),
    (dict(total_q=-8), INVALID),
    (dict(page_size=24), UNSUPPORTED),
    (dict(v=None), INVALID),
    (dict(k_pool=None), INVALID),
    (dict(v_pool=ODD), INVALID),
    (dict(block_table=None), INVALID),
    (dict(seqlens_k=None), INVALID),
    (dict(cu_seqlens_q=None), INVALID),
    (dict(max_pages=0), INVALID),
    (dict(num_pages=0), INVALID),
    (dict(num_pages=2 ** 30), UNSUPPORTED),
    (dict(v_stride=248), INVALID),
    (dict(v_pool=_Ptr((1 << 28) + 8 * 2 * 64 * 256 - 16)), INVALID),  # the end of k_pool
    (dict(k_pool=_Ptr((1 << 20) + 256)), INVALID),
    (dict(positions=_Ptr((1 << 24) + 4)), INVALID),  # inside q_out
    (dict(positions=_Ptr((1 << 28) + 4)), INVALID),  # k_pool
    (dict(positions=_Ptr((1 << 29) - 4)), INVALID),  # v_pool
])
def test_append_axes_refusals(kw, code):
    assert _append(**kw) == code
    assert attn.last_error()


def test_rows_without_tokens_are_a_no_op():
    assert _norm_rope(total=0) == attn.ATTN_OK
    assert _append(total_q=0) == attn.ATTN_OK
    assert _append(B=0) == attn.ATTN_OK


def test_pair_axis_has_an_axis_for_every_pair():
    for call in (_norm_rope, _append):
        for pairs in ([0, 1, 2], bytes(33)):
            with pytest.raises(attn.AttnError) as e:
                call(pair_axis=pairs)
            assert e.value.code == INVALID and "pair_axis" in str(e.value)


@pytest.mark.parametrize("pairs", [[0] * 31 + [1], bytes([3] * 32), [0, 1, 2, 0] * 8])
def test_pair_axis_is_looked_at_with_one_axis_too(pairs):
    for call in (_norm_rope, _append):
        assert call(axes=1, pair_axis=pairs) == INVALID and "axis" in attn.last_error()


@pytest.mark.parametrize("pairs", [np.array([0, 1, 2, 0] * 8, np.int32), np.array([0, 1, 2, 0] * 8),
                                   torch.tensor([0, 1, 2, 0] * 8), (0, 1, 2, 0) * 8,
                                   bytearray([0, 1, 2, 0] * 8)])
def test_pair_axis_of_any_whole_numbers(pairs):
    for call in (_norm_rope, _append):
        assert call(pair_axis=pairs, axes=2) == INVALID and "pair 2 goes by axis 2" in attn.last_error()


@pytest.mark.parametrize("pairs", [32, [0] * 31 + [-1], [0] * 31 + [256], [0.0] * 32, "0" * 32])
def test_pair_axis_of_anything_else_is_refused(pairs):
    for call in (_norm_rope, _append):
        with pytest.raises(attn.AttnError) as e:
            call(pair_axis=pairs)
        assert e.value.code == INVALID and "pair_axis" in str(e.value)


def _apart(names):
    return {n: _Ptr(i << 32) for i, n in enumerate(names, 1)}


def _diff(**kw):
    a = dict(B=2, Hq=4, Hkv=2, N=100, d=128, scale=0.125, mask_kind=attn.ATTN_MASK_CAUSAL, window=0,
             cu_seqlens=None, norm_weight=T, eps=1e-5, out_scale=0.8, stream=0,
             **_apart(("q", "k", "v", "o", "lse", "lam")))
    a.update(kw)
    return attn.attn_fwd_diff(**a)


def _chunk(**kw):
    a = dict(B=2, Hq=4, Hkv=2, total_q=100, d=128, scale=0.125, norm_weight=T, eps=1e-5,
             out_scale=0.8, cu_seqlens_q=T, seqlens_k=T, block_table=T, max_pages=4, page_size=64,
             num_pages=8, stream=0, **_apart(("q", "k", "v", "o", "lse", "lam")))
    a.update(kw)
    return attn.attn_fwd_diff_paged_prefill(**a)


def _decode(**kw):
    ws = attn.attn_workspace_bytes_diff(2, 4, 2, 1000, 128)
    a = dict(B=2, Hq=4, Hkv=2, N=1000, d=128, scale=0.125, norm_weight=T, eps=1e-5, out_scale=0.8,
             page_size=64, num_pages=8, workspace=_Ptr(9 << 32, n=ws), stream=0,
             **_apart(("q", "k", "v", "o", "lse", "lam", "cu_seqlens", "block_table")))
    a.update(kw)
    return attn.attn_fwd_diff_paged_decode(**a)


DIFF_REFUSALS = [
    (dict(Hq=3), INVALID),
    (dict(Hkv=0), INVALID),
    (dict(B=-1), INVALID),
    (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED),
    (dict(scale=-1.0), UNSUPPORTED),
    (dict(scale=float("inf")), INVALID),
    (dict(out_scale=float("nan")), INVALID),
    (dict(eps=-1e-6), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(q=None), INVALID),
    (dict(lam=None), INVALID),
    (dict(lse=None), INVALID),
    (dict(q=ODD), INVALID),
    (dict(o=ODD), INVALID),
    (dict(norm_weight=ODD), INVALID),
    (dict(lam=HALF), INVALID),
    (dict(o=_Ptr((1 << 32) + 2032)), INVALID),  # inside q
    (dict(o=_Ptr((2 << 32) + 16)), INVALID),
    (dict(lse=_Ptr(3 << 32)), INVALID),
    (dict(lse=_Ptr((4 << 32) + 16)), INVALID),
    (dict(o=_Ptr((6 << 32) - 2032)), INVALID),  # lam
    (dict(lse=_Ptr(6 << 32)), INVALID),
    (dict(o=_Ptr((1 << 20) + 128)), INVALID),  # norm_weight
]


@pytest.mark.parametrize("kw,code", DIFF_REFUSALS + [
    (dict(N=-1), INVALID),
    (dict(mask_kind=attn.ATTN_MASK_PAGED_DECODE), INVALID),
    (dict(mask_kind=attn.ATTN_MASK_PAGED_PREFILL), INVALID),
    (dict(mask_kind=99), INVALID),
    (dict(mask_kind=attn.ATTN_MASK_SLIDING, window=0), INVALID),
    (dict(mask_kind=attn.ATTN_MASK_PREFIX_LM, window=-1), INVALID),
    (dict(mask_kind=attn.ATTN_MASK_DOCUMENT), INVALID),  # no cu_seqlens
    (dict(mask_kind=attn.ATTN_MASK_DOCUMENT, cu_seqlens=_Ptr((4 << 32) + 64)), INVALID),  # inside o
    (dict(mask_kind=attn.ATTN_MASK_DOCUMENT, cu_seqlens=_Ptr(5 << 32)), INVALID),  # lse
    (dict(B=2 ** 30, N=2 ** 20), UNSUPPORTED),
])
def test_diff_refusals(kw, code):
    assert _diff(**kw) == code
    assert attn.last_error()


@pytest.mark.parametrize("kw,code", DIFF_REFUSALS + [
    (dict(total_q=-1), INVALID),
    (dict(page_size=8), UNSUPPORTED),
    (dict(max_pages=0), INVALID),
    (dict(num_pages=0), INVALID),
    (dict(num_pages=2 ** 30), UNSUPPORTED),
    (dict(max_pages=2 ** 26), UNSUPPORTED),
    (dict(block_table=None), INVALID),
    (dict(seqlens_k=None), INVALID),
    (dict(cu_seqlens_q=None), INVALID),
    (dict(cu_seqlens_q=_Ptr(4 << 32)), INVALID),  # o
    (dict(seqlens_k=_Ptr(5 << 32)), INVALID),  # lse
    (dict(block_table=_Ptr((5 << 32) + 64)), INVALID),
])
def test_diff_paged_prefill_refusals(kw, code):
    assert _chunk(**kw) == code
    assert attn.last_error()


@pytest.mark.parametrize("kw,code", DIFF_REFUSALS + [
    (dict(N=-1), INVALID),
    (dict(Hq=34), UNSUPPORTED),  # 17 query heads a kv head
    (dict(page_size=8), UNSUPPORTED),
    (dict(num_pages=0), INVALID),
    (dict(num_pages=2 ** 30), UNSUPPORTED),
    (dict(N=2 ** 30 + 1), UNSUPPORTED),
    (dict(B=70000), UNSUPPORTED),
    (dict(B=60000, N=2 ** 29), UNSUPPORTED),  # more blocks than an int counts
    (dict(block_table=None), INVALID),
    (dict(cu_seqlens=None), INVALID),
    (dict(workspace=None), WORKSPACE),
    (dict(workspace=_Ptr(9 << 32, n=1024)), WORKSPACE),
    (dict(o=_Ptr((6 << 32) - 2032)), INVALID),  # lam
    (dict(o=_Ptr((7 << 32) - 2032)), INVALID),  # cu_seqlens
    (dict(lse=_Ptr(8 << 32)), INVALID),
    (dict(o=_Ptr((9 << 32) + 4096)), INVALID),  # the workspace
    (dict(v=_Ptr((9 << 32) - 16)), INVALID),
    (dict(N=0, o=None), INVALID),
    (dict(N=0, lse=ODD), INVALID),
    (dict(N=0, cu_seqlens=None), INVALID),
])
def test_diff_paged_decode_refusals(kw, code):
    assert _decode(**kw) == code
    assert attn.last_error()


def test_nothing_to_do_is_a_no_op():
    assert _diff(B=0) == attn.ATTN_OK and _diff(N=0) == attn.ATTN_OK
    assert _chunk(B=0) == attn.ATTN_OK and _chunk(total_q=0) == attn.ATTN_OK
    assert _decode(B=0) == attn.ATTN_OK


def test_diff_workspace():
    need = attn.attn_workspace_bytes_diff(32, 32, 8, 16384, 128)
    assert need > 0 and need % 256 == 0
    assert attn.attn_workspace_bytes_diff(1, 32, 8, 131072, 128) == need
    assert attn.attn_workspace_bytes_diff(32, 64, 8, 16384, 128) > need
    assert attn.attn_workspace_bytes_diff(0, 32, 8, 128, 128) == 0
    assert attn.attn_workspace_bytes_diff(1, 32, 8, 128, 96) == 0


CALLS = [lambda t, **kw: _norm_rope(q=t, k=t, q_out=t, k_out=t, cos_sin=t, positions=t, **kw),
         lambda t, **kw: _append(**{n: t for n in ("q", "k", "v", "q_out", "k_pool", "v_pool",
                                                   "cos_sin", "positions", "cu_seqlens_q",
                                                   "seqlens_k", "block_table")}, **kw),
         lambda t, **kw: _diff(q=t, k=t, v=t, o=t, lse=t, lam=t, norm_weight=t, **kw),
         lambda t, **kw: _chunk(q=t, k=t, v=t, o=t, lse=t, lam=t, norm_weight=t, cu_seqlens_q=t,
                                seqlens_k=t, block_table=t, **kw),
         lambda t, **kw: _decode(q=t, k=t, v=t, o=t, lse=t, lam=t, norm_weight=t, cu_seqlens=t,
                                 block_table=t, workspace=t, **kw)]


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors_are_refused(call):
    with pytest.raises(attn.AttnError) as e:
        call(_Ptr(device=-1))
    assert e.value.code == INVALID and "host memory" in str(e.value)


@pytest.mark.parametrize("call", CALLS)
def test_another_device_than_the_current_one_is_refused(call, monkeypatch):
    monkeypatch.setattr(attn, "_launch_device", lambda: 0)
    with pytest.raises(attn.AttnError) as e:
        call(_Ptr(device=1))
    assert e.value.code == INVALID and "[0, 1]" in str(e.value)


# ------------------------------------------------------------------ the oracle's own pins

def test_one_axis_is_the_ordinary_rotation():
    rng = np.random.default_rng(1)
    x, cs = rng.standard_normal((5, 3, 64)), rng.standard_normal((9, 48))
    pos = rng.integers(0, 9, 5)
    for il in (False, True):
        want = cache.rotate(x, cs, pos, 48, il)
        got, _ = diff.prepare(x, 1, None, 0, cs, pos[None], [0] * 24, 48, il)
        np.testing.assert_allclose(got, want, atol=1e-14)
        three = np.stack([pos + 1, pos, pos + 2]) % 9
        got, _ = diff.prepare(x, 1, None, 0, cs, three, [1] * 24, 48, il)
        np.testing.assert_allclose(got, cache.rotate(x, cs, three[1], 48, il), atol=1e-14)


def test_two_maps_are_two_heads():
    rng = np.random.default_rng(2)
    x, cs = rng.standard_normal((5, 3, 64)), rng.standard_normal((9, 32))
    pos, w = rng.integers(0, 9, (2, 5)), rng.standard_normal(32)
    axis = [0, 1] * 8
    got, _ = diff.prepare(x, 2, w, 1e-6, cs, pos, axis, 32, False)
    want, _ = diff.prepare(x.reshape(5, 6, 32), 1, w, 1e-6, cs, pos, axis, 32, False)
    np.testing.assert_allclose(got.reshape(5, 6, 32), want, atol=1e-14)


def test_diff_rows_pins():
    """lam = 0 is the first map's attention, equal maps cancel to 1 - lam of it, a window of one is
    (1 - lam) v, and a row of nothing is zero."""
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((h, 7, 64)) for h in (4, 2, 2))
    here = diff.visible("causal", 0, 7)
    one = diff.Rows(q, k, v, here, np.zeros(4), 0.2, None, 0, 1.0)
    for h in range(4):
        s = np.where(here, q[h][:, :32] @ k[h // 2][:, :32].T * 0.2, -np.inf)
        w = np.exp(s) / np.exp(s).sum(1, keepdims=True)
        np.testing.assert_allclose(one.o[h], w @ v[h // 2], atol=1e-12)
        np.testing.assert_allclose(one.lse[h, 0], np.log(np.exp(s).sum(1)), atol=1e-12)
    q2, k2 = (np.concatenate([a[..., :32]] * 2, -1) for a in (q, k))
    same = diff.Rows(q2, k2, v, here, np.full(4, 0.25), 0.2, None, 0, 1.0)
    np.testing.assert_allclose(same.o, 0.75 * one.o, atol=1e-12)
    near = diff.Rows(q, k, v, diff.visible("sliding", 1, 7), np.full(4, 0.25), 0.2, None, 0, 2.0)
    np.testing.assert_allclose(near.o, 1.5 * np.repeat(v, 2, 0), atol=1e-12)
    w = rng.standard_normal(64)
    normed = diff.Rows(q, k, v, here, np.full(4, 0.25), 0.2, w, 1e-5, 1.0)
    free = diff.Rows(q, k, v, here, np.full(4, 0.25), 0.2, None, 0, 1.0)
    np.testing.assert_allclose(normed.o, cache.norm(free.o, w, 1e-5), atol=1e-12)
    none = diff.Rows(q, k, v, np.zeros((7, 7), bool), np.ones(4), 0.2, w, 0.0, 1.0)
    assert (none.o == 0).all() and (none.lse == -np.inf).all() and (none.o_tol < 1e-30).all()


@pytest.mark.parametrize("n", [145, 641, 1900])
@pytest.mark.parametrize("normed", [False, True])
def test_two_norm_bounds_catch_small_mistakes(n, normed):
    """Blocks of 64 rows with lam, the norm's eps or weights rounded wrong are outside the bound; the
    same rows with P and the output rounded to bf16 inside."""
    rng = np.random.default_rng(n)
    d, rows = 64, 64
    q, k, v = rng.standard_normal((1, rows, d)), rng.standard_normal((1, n, d)), rng.standard_normal(
        (1, n, d))
    here, lam, scale = np.ones((rows, n), bool), np.array([0.6]), 32 ** -0.5
    w = 1 + 0.3 * rng.standard_normal(d) if normed else None
    want, bound = diff.two_norm(q, k, v, here, lam, scale, w, 1e-5, 0.8)
    assert bound.sum() <= 2.0 ** -14 * (want ** 2).sum()

    def bf16(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()

    def run(lam=0.6, drop=0, cut=lambda x: x):
        y = 0
        for m, f in ((0, 1.0), (1, -lam)):
            s = q[0][:, 32 * m:32 * m + 32] @ k[0][:, 32 * m:32 * m + 32].T * scale
            p = np.exp(s - s.max(1, keepdims=True))
            y = y + f * ((cut(p)[:, drop:] @ v[0][drop:]) / p.sum(1, keepdims=True))
        if normed:
            y = y / np.sqrt((y * y).mean(1, keepdims=True) + 1e-5) * w
        return 0.8 * y

    def inside(o):
        return ((o - want[0]) ** 2).sum() <= bound.sum()

    assert inside(bf16(run(cut=bf16)))
    for o in (run(lam=0.62), run(drop=1), run(cut=lambda x: bf16(x) * 1.02) if not normed else
              run(lam=0.58), run(cut=lambda x: np.floor(x * 32) / 32)):
        assert not inside(bf16(o))


def _cases():
    path = os.path.join(ROOT, "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operators_under_test", path)
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    return ops


def test_plain_forms_agree_with_the_oracle():
    """perf/more_operators.py's 32-bit rows and its count of visible pairs against the oracle's."""
    ops = _cases()
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(h, 9, 64, generator=gen) for h in (2, 1, 1))
    s = {"d": 64, "scale": 0.3, "weight": torch.rand(64, generator=gen)}
    lam = np.array([0.4, -0.3])
    for mask in ("none", "causal", "sliding", "sliding_bidir", "prefix"):
        case = {"mask": mask, "window": 3}
        here = diff.visible(mask, 3, 9)
        assert ops._seen(case, 9) == here.sum()
        o, lse = ops._plain_rows(s, q, k, v, torch.from_numpy(here), torch.tensor(lam).view(2, 1, 1))
        want = diff.Rows(q.double().numpy(), k.double().numpy(), v.double().numpy(), here, lam, 0.3,
                         s["weight"].numpy(), ops.EPS, ops.OUT_SCALE)
        np.testing.assert_allclose(o.numpy(), want.o, atol=2e-5)
        np.testing.assert_allclose(lse.numpy(), want.lse, atol=2e-6)
