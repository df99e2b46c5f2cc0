"""Blocks of few rows over the 8-bit cache, in every order in which the streams may
come to take them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda

from .test_paged_attention_quant_gpu import BF16, FP16, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("pattern", ["keys nothing keys keys", "pages given up", "any"])
def test_single_tokens_among_requests_without_keys(pattern, dtype):
    """Requests without cached tokens take a turn of the streams without a block, so that one stream
    leads several blocks in a row; pages that have been given up have no copies to wait for, so
    that keys are there before queries.  Every run gives the same bits."""
    r = np.random.default_rng(len(pattern))
    n = 1200
    if pattern == "keys nothing keys keys":
        kv = [int(x) for _ in range(n // 4) for x in (r.integers(1, 300), 0, r.integers(1, 300), r.integers(1, 40))]
        gone = [i % 8 == 0 for i in range(n)]
    elif pattern == "pages given up":
        kv = [0 if i % 5 == 1 else int(r.integers(1, 300)) for i in range(n)]
        gone = [i % 5 != 4 for i in range(n)]
    else:
        kv = [int(x) for x in r.integers(1, 300, n) * (r.random(n) < 0.7)]
        gone = (r.random(n) < 0.4).tolist()
    c = Case([1] * n, kv, 4, 2, 16, dtype, seed=n)
    c.table = [[-1] * len(row) if x else row for row, x in zip(c.table, gone)]
    first = c.run()
    c.check(result=first)
    ws = kda.paged_attention_workspace(tokens=n, heads=4)
    for _ in range(20):
        again = c.run(workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert kda.kda_device_status() == 0 and not ws[:4096].any()
