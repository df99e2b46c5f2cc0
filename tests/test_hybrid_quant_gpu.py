"""The hybrid model's serving steps with rotary positions and a cache in 8 bits:
rope, append and attention among recurrent layers, drafts rolled back, pages
handed back.  (The example's own run is tested with the 16-bit cache.)"""
from __future__ import annotations

import os
import sys

import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("window,sinks", [(0, 0), (96, 4)])
def test_steps_run_and_leave_nothing_behind(window, sinks):
    import hybrid_serving as ex

    r = torch.Generator().manual_seed(3)
    texts = [torch.randint(512, (n,), generator=r).tolist() for n in (9, 40, 73, 137, 200, 300)]
    rope = kda.Rope(kda.rope_frequencies(128, 5e5, factor=4.0, original_context=256))
    model = ex.HybridModel(window=window, sinks=sinks, rope=rope, quantized=True, requests=6)
    first = ex.serve(model, texts, 128)
    assert all(torch.isfinite(x).all() and x.shape == (len(t), 512) for x, t in zip(first, texts))
    assert int(model.pages.free_count) == 64 and not model.pages.kv_lens.any() and kda.kda_device_status() == 0
    again = ex.serve(ex.HybridModel(window=window, sinks=sinks, rope=rope, quantized=True, requests=6), texts, 128)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
