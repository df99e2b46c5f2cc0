"""What the hybrid model's layers hand to rope, append and attention, step by step,
and what comes back, against positions, lengths and cached tokens that the test
keeps for itself: prompt chunks, a rejected draft, single tokens."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from oracle import quant

from .test_paged_attention_quant_gpu import BF16, Case, _np

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_every_step_of_the_attention_layers(window, sinks, monkeypatch):
    import hybrid_serving as ex

    heads, kv_heads, n_req = 8, 2, 4
    f = kda.rope_frequencies(128, 5e5, factor=4.0, original_context=64)
    state = dict(lens=[0] * n_req, new=None, turned=0, attended=0)
    history = [[[], []] for _ in range(n_req)]  # keys and values of every token, in 64 bits
    case = Case([1], [1], heads, kv_heads, 16)  # for its check
    rope, append, attend = kda.kda_rope, kda.kda_kv_append, kda.kda_paged_attention

    def positions():
        return [n + i for n, new in zip(state["lens"], state["new"]) for i in range(new)]

    def checked_rope(handle, q, k, **kw):
        raw = _np(q), _np(k)
        got = rope(handle, q, k, **kw)
        assert got[0] is q and got[1] is k
        for x, y in zip(raw, got):
            want = quant.rope(x, positions(), f.tolist())
            size = np.tile(np.hypot(x[..., :64], x[..., 64:]), 2)  # of each pair
            # rounded once to bf16; products, sum, cosine and sine in 32 bits
            assert (np.abs(_np(y) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size).all()
        state["turned"] += 1
        return got

    def checked_append(cache, k, v, slots, **kw):
        append(cache, k, v, slots, **kw)
        at = 0
        for b, new in enumerate(state["new"]):
            for x, tokens in zip((k, v), history[b]):
                tokens[state["lens"][b]:] = list(_np(x)[at:at + new])
            at += new

    def checked_attention(cache, q, cu, kv_lens, table, **kw):
        out, lse = attend(cache, q, cu, kv_lens, table, return_lse=True, **kw)
        case.k, case.v, case.ks, case.vs, case.q = cache.k, cache.v, cache.k_scale, cache.v_scale, q
        case.page, case.scale, case.dtype = cache.k.shape[1], 128 ** -0.5, BF16
        case.cu = np.concatenate([[0], np.cumsum(state["new"])]).tolist()
        case.kv = [n + new for n, new in zip(state["lens"], state["new"])]
        case.table = table.tolist()
        assert kw["window"] == window and kw["sinks"] == sinks
        case.check(window, sinks, result=(out, lse))
        for b in range(n_req):
            where = tuple(np.array(case.rows(b)).T) if case.kv[b] else None
            for number, scale, tokens in zip(case.numbers(), (cache.k_scale, cache.v_scale), history[b]):
                if where is None:
                    continue
                want = np.stack(tokens)
                step = _np(scale)[where[0], :, where[1] // 16][..., None] * 2.0 ** -10
                # half a step of 4 bits, or half of the least step, the latter once more where the scale has grown
                assert (np.abs(number[where] - want) <= np.maximum(2.0 ** -4 * np.abs(want), step) + step).all()
        state["attended"] += 1
        return out, lse

    class Model(ex.HybridModel):
        def step(self, tokens, new_lens):
            state["new"] = list(new_lens)
            got = super().step(tokens, new_lens)
            state["lens"] = [n + new for n, new in zip(state["lens"], new_lens)]
            return got

        def rollback(self, keep_lens):
            super().rollback(keep_lens)
            state["lens"] = [min(n, k) for n, k in zip(state["lens"], keep_lens)]

    for name, call in (("kda_rope", checked_rope), ("kda_kv_append", checked_append), ("kda_paged_attention", checked_attention)):
        monkeypatch.setattr(ex.kda, name, call)
    model = Model(window=window, sinks=sinks, requests=n_req, rope=kda.Rope(f), quantized=True, page_size=16)
    r = torch.Generator().manual_seed(3)
    ex.serve(model, [torch.randint(512, (n,), generator=r).tolist() for n in (9, 40, 73, 137)], 50)
    assert state["turned"] == state["attended"] > 8 and state["lens"] == [0] * n_req
    assert int(model.pages.free_count) == 64 and kda.kda_device_status() == 0
