"""Ordinary prefill whose last 128-row tiles hold whole warps past the prompt's end, with many units a
CTA: every row against the oracle, and the same bits each time."""
import pytest
import torch

from tiled_attention_gb300 import inputs as I
from test_gpu_parity import compare, cuda_library, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [257, 300, 417, 385])
@pytest.mark.parametrize("mask,window", [(I.MASK_NONE, 0), (I.MASK_CAUSAL, 0), (I.MASK_SLIDING, 150),
                                         (I.MASK_SLIDING_BIDIR, 90)])
def test_last_tiles_of_many_units(d, N, mask, window):
    w = I.dense_workload(N + d, 12, 32, 8, N, d, mask, window)
    dp = run(w)
    compare(w, dp, strict=False)
    o, lse = dp.o.view(torch.int16).clone(), dp.lse.clone()
    for _ in range(5):
        dp.o.fill_(float("nan"))
        assert dp.run() == 0
        torch.cuda.synchronize()
        assert torch.equal(dp.o.view(torch.int16), o) and torch.equal(dp.lse, lse)
