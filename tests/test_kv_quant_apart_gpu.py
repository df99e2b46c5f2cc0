"""The 8-bit cache's append where tokens of one block stand apart: the first of them
are written, the others reported and left out, every time alike."""
from __future__ import annotations

import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from oracle import quant

from .test_kv_quant_gpu import BF16, FP16, INDEX, Pool, _i32, _np

pytestmark = pytest.mark.gpu


def _far(n):
    """n tokens of other blocks, from slot 64 on"""
    return list(range(64, 64 + n))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("slots,left_out", [
    ([5, -1, 6], [2]),  # a token skipped
    ([5, 6, -1, -1, 8, 9, 10], [4, 5, 6]),
    ([5, 40, 6], [2]),  # another request's token between
    ([0, 1] + _far(30) + [2, 3], [32, 33]),  # 31 tokens on
    ([0, 1] + _far(31) + [2], [33]),  # 32 tokens on
    ([5, -1, 6] + _far(31) + [7], [2, 34]),  # near to one that was left out
    ([17] + _far(14) + [18, 19, 20, 21, 22, 23, 24, 25, 26, 27, 28, 29, 30, 31, 32, 33], list(range(15, 29))),  # and on to the next block
    ([3, -1, 1], [2]),  # backwards
])
def test_tokens_of_a_block_that_stand_apart(slots, left_out, dtype):
    for _ in range(5):
        p = Pool(16, 16, 2, dtype, seed=len(slots))
        k, v = p.rows(len(slots), gain=3.0, seed=2)
        kda.kda_kv_append(p.cache, k, v, _i32(slots))
        assert kda.kda_device_status() == INDEX
        kept = [-1 if i in left_out else s for i, s in enumerate(slots)]
        for i, x in ((0, k), (2, v)):
            quant.append(p.want[i], p.want[i + 1], _np(x), kept)
        p.same()


def test_a_long_prompt_with_a_token_skipped():
    """Where a warp looks for blocks among many tokens."""
    n = 160 * 1024 // 2
    p = Pool(n // 64 + 2, 64, 1, seed=3)
    slots = list(range(n))
    slots[40] = slots[5000 * 16 - 1] = slots[n - 32] = -1  # within a block, at the end of one, at the start of one
    k, v = p.rows(n, seed=4)
    kda.kda_kv_append(p.cache, k, v, _i32(slots))
    assert kda.kda_device_status() == INDEX
    kept = [-1 if 40 <= i < 48 else s for i, s in enumerate(slots)]
    for i, x in ((0, k), (2, v)):
        quant.append(p.want[i], p.want[i + 1], _np(x), kept)
    p.same()


def test_neighbours_in_other_blocks_are_no_hindrance():
    p = Pool(40, 16, 2, seed=5)
    slots = [b * 16 + (7 * b) % 16 for b in range(40)]
    p.append(*p.rows(40, seed=6), slots)
    p.append(*p.rows(40, seed=7), [s - 1 if s % 16 else s for s in slots])
    p.append(*p.rows(3, seed=8), [0, 16, 32])
    p.same()
    assert kda.kda_device_status() == 0 and torch.isfinite(p.cache.k_scale).all()
