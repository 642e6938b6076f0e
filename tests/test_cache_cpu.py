"""The cache entry points' argument checks (before any CUDA call) and the 4-bit oracle's own
pins. CPU only."""
import numpy as np
import pytest
import torch

from oracle import cache
from tiled_attention_gb300 import attn, build

INVALID, UNSUPPORTED, WORKSPACE = (attn.ATTN_ERR_INVALID, attn.ATTN_ERR_UNSUPPORTED,
                                   attn.ATTN_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()
    return attn.lib()


class _Ptr:
    """Stands in for a device tensor in calls that fail validation: never dereferenced."""

    def __init__(self, addr=1 << 20, device=0):
        self.addr, self.device = addr, device

    def data_ptr(self):
        return self.addr

    def get_device(self):
        return self.device


T = _Ptr()
OUT, OUT2 = _Ptr(1 << 24), _Ptr(1 << 25)  # outputs apart from the inputs
ODD = _Ptr((1 << 20) | 8)


def _norm_rope(**kw):
    a = dict(q=T, k=T, q_out=OUT, k_out=OUT2, total=8, N=4, Hq=4, Hkv=2, d=128, q_stride=512,
             k_stride=256, q_weight=None, k_weight=None, eps=1e-6, cos_sin=T, max_pos=16,
             rot_dim=128, interleaved=False, positions=None, stream=0)
    a.update(kw)
    return attn.attn_norm_rope(**a)


ROW_REFUSALS = [
    (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED),
    (dict(rot_dim=-16), INVALID),
    (dict(rot_dim=144), INVALID),
    (dict(rot_dim=24), UNSUPPORTED),
    (dict(max_pos=0), INVALID),
    (dict(cos_sin=None), INVALID),
    (dict(cos_sin=ODD), INVALID),
    (dict(q=ODD), INVALID),
    (dict(k=ODD), INVALID),
    (dict(q_out=None), INVALID),
    (dict(q_out=ODD), INVALID),
    (dict(q_stride=504), INVALID),  # below the heads' width
    (dict(q_stride=516), INVALID),  # rows not 16-byte aligned
    (dict(k_stride=-256), INVALID),
    (dict(q_weight=ODD), INVALID),
    (dict(k_weight=T, eps=float("nan")), INVALID),
    (dict(q_weight=T, eps=-1.0), INVALID),
    (dict(N=0), INVALID),
    (dict(q_out=T), INVALID),  # in place
    (dict(q_out=_Ptr((1 << 20) + 7 * 1024)), INVALID),  # into the last row
]


@pytest.mark.parametrize("kw,code", ROW_REFUSALS + [
    (dict(total=-1), INVALID),
    (dict(total=9), INVALID),  # not rows of N
    (dict(k_out=None), INVALID),
    (dict(k_out=ODD), INVALID),
    (dict(q=None, k=None), INVALID),
    (dict(Hq=-1), INVALID),
    (dict(Hq=0, Hkv=0), INVALID),
    (dict(k_out=_Ptr((1 << 20) + 256)), INVALID),
    (dict(max_pos=3), INVALID),  # rows of 4 positions, a table of 3
])
def test_norm_rope_refusals(kw, code):
    assert _norm_rope(**kw) == code
    assert attn.last_error()


FAR = _Ptr(1 << 30)


@pytest.mark.parametrize("call", [
    lambda: _norm_rope(k_out=_Ptr((1 << 24) + 4096)),  # outputs into one another
    lambda: _append(False, k_pool=FAR, v_pool=FAR),
    lambda: _append(True, k_pool=FAR, v_pool=FAR),
    # K's pool: 8 pages x 2 heads x 16 tokens of 256 or 72 bytes; V's begins in its last row
    lambda: _append(False, k_pool=FAR, v_pool=_Ptr((1 << 30) + 256 * 255)),
    lambda: _append(True, k_pool=FAR, v_pool=_Ptr((1 << 30) + 72 * 254)),
    lambda: _append(False, k_pool=OUT, v_pool=FAR),  # q_out
    lambda: _append(True, k_pool=FAR, v_pool=OUT),
    lambda: _append(False, k_pool=T, v_pool=FAR),  # an input
    lambda: _append(True, k_pool=FAR, v_pool=T),
    lambda: _unpack(),
    lambda: _unpack(dst=FAR, pool=_Ptr((1 << 30) + 2 * 4 * 2 * 16 * 256 - 16)),
    lambda: _unpack(pool=FAR, dst=_Ptr((1 << 30) + 8 * 2 * 16 * 72 - 16)),
])
def test_overlapping_outputs_are_refused(call):
    assert call() == INVALID
    assert "overlap" in attn.last_error()


def test_norm_rope_without_tokens_is_a_no_op():
    assert _norm_rope(total=0) == attn.ATTN_OK
    assert _norm_rope(total=0, q=None, k=None, cos_sin=None) == attn.ATTN_OK


def _append(fp4, **kw):
    a = dict(q=T, k=T, v=T, q_out=OUT, k_pool=T, v_pool=T, B=2, Hq=4, Hkv=2, total_q=8, N=8, d=128,
             q_stride=512, k_stride=256, v_stride=256, q_weight=None, k_weight=None, eps=1e-6,
             cos_sin=T, max_pos=64, rot_dim=128, interleaved=False, cu_seqlens_q=T, seqlens_k=T,
             block_table=T, max_pages=4, page_size=16, num_pages=8, stream=0)
    if fp4:
        a.update(k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return (attn.attn_append_paged_fp4 if fp4 else attn.attn_append_paged)(**a)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("kw,code", ROW_REFUSALS + [
    (dict(total_q=-8), INVALID),
    (dict(total_q=12), INVALID),
    (dict(B=-1), INVALID),
    (dict(Hkv=0), INVALID),
    (dict(k=None), INVALID),
    (dict(v=None), INVALID),
    (dict(v=ODD), INVALID),
    (dict(v_stride=128), INVALID),
    (dict(k_pool=None), INVALID),
    (dict(v_pool=ODD), INVALID),
    (dict(cu_seqlens_q=None), INVALID),
    (dict(seqlens_k=None), INVALID),
    (dict(block_table=None), INVALID),
    (dict(max_pages=0), INVALID),
    (dict(num_pages=0), INVALID),
    (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED),
    (dict(num_pages=2 ** 30), UNSUPPORTED),
    (dict(max_pages=2 ** 28), UNSUPPORTED),
])
def test_append_refusals(fp4, kw, code):
    assert _append(fp4, **kw) == code
    assert attn.last_error()


@pytest.mark.parametrize("fp4", [False, True])
def test_append_without_tokens_is_a_no_op(fp4):
    assert _append(fp4, B=0) == attn.ATTN_OK
    assert _append(fp4, total_q=0) == attn.ATTN_OK


@pytest.mark.parametrize("kw,code", [
    (dict(k_scale=0.0), INVALID),
    (dict(v_scale=-1.0), INVALID),
    (dict(k_scale=float("inf")), INVALID),
    (dict(v_scale=float("nan")), INVALID),
    (dict(k_scale=1e-39), INVALID),  # no finite reciprocal
    (dict(rot_dim=16), UNSUPPORTED),  # half-split pairs would cut 16-channel blocks
])
def test_append_fp4_refusals(kw, code):
    assert _append(True, **kw) == code
    assert attn.last_error()


def _unpack(**kw):
    a = dict(pool=T, dst=T, pool_scale=1.0, block_table=T, seqlens=T, B=2, max_pages=4, Hkv=2,
             page_size=16, d=128, num_pages=8, stream=0)
    a.update(kw)
    return attn.attn_unpack_pages_fp4(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(d=32), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED),
    (dict(pool_scale=0.0), INVALID),
    (dict(pool_scale=float("nan")), INVALID),
    (dict(pool=None), INVALID),
    (dict(dst=ODD), INVALID),
    (dict(seqlens=None), INVALID),
    (dict(block_table=None), INVALID),
    (dict(B=-1), INVALID),
    (dict(Hkv=0), INVALID),
    (dict(B=70000), UNSUPPORTED),
    (dict(max_pages=2 ** 28), UNSUPPORTED),
])
def test_unpack_refusals(kw, code):
    assert _unpack(**kw) == code
    assert attn.last_error()


def test_unpack_nothing_is_a_no_op():
    assert _unpack(B=0) == attn.ATTN_OK
    assert _unpack(max_pages=0) == attn.ATTN_OK


def _decode(**kw):
    a = dict(q=T, k=T, v=T, o=T, lse=T, B=2, Hq=4, Hkv=2, N=100000, d=128, scale=0.1,
             k_scale=1.0, v_scale=1.0, cu_seqlens=T, block_table=T, page_size=64, num_pages=8,
             workspace=None, stream=0)
    a.update(kw)
    return attn.attn_fwd_paged_decode_fp4(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3), INVALID),
    (dict(Hq=34), UNSUPPORTED),  # 17 query heads a kv head
    (dict(d=96), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED),
    (dict(scale=-1.0), UNSUPPORTED),
    (dict(scale=float("inf")), INVALID),
    (dict(k_scale=0.0), INVALID),
    (dict(v_scale=-2.0), INVALID),
    (dict(k_scale=float("nan")), INVALID),
    (dict(scale=1e30, k_scale=1e30), INVALID),
    (dict(cu_seqlens=None), INVALID),
    (dict(block_table=None), INVALID),
    (dict(num_pages=0), INVALID),
    (dict(num_pages=2 ** 30), UNSUPPORTED),
    (dict(N=2 ** 30 + 1), UNSUPPORTED),
    (dict(q=ODD), INVALID),
    (dict(k=ODD), INVALID),
    (dict(B=70000), UNSUPPORTED),
    (dict(B=60000, N=2 ** 29), UNSUPPORTED),  # more blocks than an int counts
    (dict(B=-1), INVALID),
    (dict(), WORKSPACE),
])
def test_decode_fp4_refusals(kw, code):
    assert _decode(**kw) == code
    assert attn.last_error()


def test_decode_fp4_empty_is_a_no_op():
    assert _decode(B=0) == attn.ATTN_OK
    assert _decode(N=0) == attn.ATTN_OK


class _Bytes(_Ptr):
    """A stand-in with a size, for the workspace."""

    def __init__(self, addr, n):
        super().__init__(addr)
        self.n = n

    def numel(self):
        return self.n

    def element_size(self):
        return 1


def _decode_apart(**kw):
    """A decode whose tensors lie apart: q, K, V, o, lse, cu, table and the workspace at 1 to 8
    times 4 GB. B = 2, Hq = 4, Hkv = 2, d = 128, 8 pages of 64: q and o 2048 bytes, lse 32,
    pools 73728, cu 12, the table's 1563 columns 12504."""
    ws = attn.attn_workspace_bytes_fp4(2, 4, 2, 100000, 128)
    a = {n: _Ptr(i << 32) for i, n in enumerate(("q", "k", "v", "o", "lse", "cu_seqlens",
                                                 "block_table"), 1)}
    a["workspace"] = _Bytes(8 << 32, ws)
    a.update(kw)
    return _decode(**a)


@pytest.mark.parametrize("kw", [
    dict(o=_Ptr(1 << 32)),  # q's place
    dict(o=_Ptr((1 << 32) + 2032)),  # the end of q
    dict(lse=_Ptr((1 << 32) + 1024)),
    dict(lse=_Ptr((1 << 32) - 16)),
    dict(o=_Ptr((2 << 32) + 73712)),  # the end of K
    dict(lse=_Ptr(3 << 32)),
    dict(lse=_Ptr((4 << 32) + 2032)),  # the end of o
    dict(o=_Ptr(5 << 32)),
    dict(o=_Ptr((6 << 32) - 2032)),  # cu_seqlens
    dict(lse=_Ptr((7 << 32) + 12496)),  # the end of the table
    dict(q=_Ptr((8 << 32) + 4096)),  # the workspace
    dict(o=_Ptr((8 << 32) + 4096)),
    dict(lse=_Ptr((8 << 32) - 16)),
    dict(v=_Ptr((8 << 32) - 73712)),
    dict(block_table=_Ptr((8 << 32) - 12496)),
])
def test_decode_fp4_overlaps_are_refused(kw):
    assert _decode_apart(**kw) == INVALID
    assert "overlap" in attn.last_error()


@pytest.mark.parametrize("kw", [dict(o=None), dict(lse=None), dict(cu_seqlens=None), dict(o=ODD)])
def test_decode_fp4_without_keys_still_has_rows_to_write(kw):
    """N = 0: the sequences are empty, but their rows and lengths are there."""
    assert _decode(N=0, **kw) == INVALID
    assert attn.last_error()


def test_decode_fp4_workspace():
    need = attn.attn_workspace_bytes_fp4(32, 32, 8, 16384, 128)
    # two partial rows of 4 heads a resident CTA, O and (max, sum): the batch and the contexts
    # do not matter, the group does
    assert need > 0 and need % 256 == 0
    assert attn.attn_workspace_bytes_fp4(1, 32, 8, 131072, 128) == need
    assert attn.attn_workspace_bytes_fp4(32, 64, 8, 16384, 128) > need
    assert attn.attn_workspace_bytes_fp4(0, 32, 8, 128, 128) == 0
    assert attn.attn_workspace_bytes_fp4(1, 32, 8, 128, 96) == 0


def test_tensors_of_two_devices_are_refused():
    far = _Ptr(device=1)
    for call in (lambda: _norm_rope(k_out=far), lambda: _append(False, block_table=far),
                 lambda: _append(True, v_pool=far), lambda: _unpack(seqlens=far),
                 lambda: _decode(lse=far)):
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.code == INVALID and "device" in str(e.value)


CALLS = [lambda t, **kw: _norm_rope(q=t, k=t, q_out=t, k_out=t, cos_sin=t, **kw),
         lambda t, **kw: _append(False, **_rows_on(t), **kw),
         lambda t, **kw: _append(True, **_rows_on(t), **kw),
         lambda t, **kw: _unpack(pool=t, dst=t, block_table=t, seqlens=t, **kw),
         lambda t, **kw: _decode(q=t, k=t, v=t, o=t, lse=t, cu_seqlens=t, block_table=t, **kw)]


def _rows_on(t):
    return {n: t for n in ("q", "k", "v", "q_out", "k_pool", "v_pool", "cos_sin", "cu_seqlens_q",
                           "seqlens_k", "block_table")}


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors_are_refused_on_a_given_stream_too(call):
    """All of a call's tensors in host memory are of one device, but not of one to launch on."""
    with pytest.raises(attn.AttnError) as e:
        call(_Ptr(device=-1), stream=0)
    assert e.value.code == INVALID and "host memory" in str(e.value)


class _Stream:
    cuda_stream = 0

    def __init__(self, device_index):
        self.device_index = device_index


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("tensors,stream", [(1, 0), (1, _Stream(1)), (1, _Stream(0)),
                                            (0, _Stream(1))])
def test_another_device_than_the_current_one_is_refused(call, tensors, stream, monkeypatch):
    """The library launches on the current device, here 0, whatever the stream is."""
    monkeypatch.setattr(attn, "_launch_device", lambda: 0)
    with pytest.raises(attn.AttnError) as e:
        call(_Ptr(device=tensors), stream=stream)
    assert e.value.code == INVALID and "[0, 1]" in str(e.value)


# ------------------------------------------------------------------ the oracle's own pins

def test_e2m1_rounding():
    x = np.array([0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 7, 100])
    want = [0, 1, 2, 1, 2, 3, 4, 4, 5, 6, 6, 7, 7, 7]
    assert cache.e2m1_round(x).tolist() == want
    assert cache.e2m1_round(-x).tolist() == [w + 8 for w in want]
    assert cache.e2m1_round(np.array([0.0, -0.0])).tolist() == [0, 8]


def test_quantize_values_error():
    """A value is off by at most half of the widest code step at its block's scale: 1 * scale,
    or the saturation of 6 / (1 - 2^-4) to 6 where the scale rounded down, 0.4 * scale."""
    rng = np.random.default_rng(3)
    y = (rng.standard_normal((50, 2, 128)) * np.exp(rng.uniform(-1, 4, (50, 2, 1)))).astype(
        np.float32)
    for g in (1.0, 0.125, 0.3):
        codes, sf = cache.quantize(y, g)
        got = cache.values(codes, sf, g)
        step = np.repeat(cache._E4M3[sf], 16, axis=-1) * g
        assert np.all(np.abs(got - y) <= step * (1 + 1e-6))
        rel = np.linalg.norm(got - y) / np.linalg.norm(y)
        assert rel < 0.2


def test_rotation_turns_pairs():
    """A turn keeps each pair's length; two turns add their angles."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 2, 64))
    ang = rng.uniform(-3, 3, (5, 16))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], axis=1)
    two = np.concatenate([np.cos(2 * ang), np.sin(2 * ang)], axis=1)
    pos = np.array([4, 0, 2])
    for il in (False, True):
        y = cache.rotate(x, cs, pos, 32, il)
        a, b = cache.pairs(32, il)
        np.testing.assert_allclose(np.hypot(y[..., a], y[..., b]), np.hypot(x[..., a], x[..., b]))
        np.testing.assert_allclose(cache.rotate(y, cs, pos, 32, il),
                                   cache.rotate(x, two, pos, 32, il), atol=1e-12)
        assert np.array_equal(y[..., 32:], x[..., 32:])


def test_plain_forms_agree_with_the_oracle():
    """perf/operators.py's 32-bit quantizer and value table against the oracle's."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf",
                        "operators.py")
    spec = importlib.util.spec_from_file_location("operators_under_test", path)
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    x = torch.randn(7, 3, 128, generator=torch.Generator().manual_seed(1)) * 3
    codes, sf = ops._quantize(x, 0.5)
    want, wsf = cache.quantize(x.numpy(), 0.5)
    assert np.array_equal(sf.numpy(), wsf)
    got = cache.values(codes.numpy(), sf.numpy(), 0.5)
    assert np.array_equal(got, cache.values(want, wsf, 0.5))
