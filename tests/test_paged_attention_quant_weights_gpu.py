"""Weights over the 8-bit cache are fp16 numbers, all of each, in blocks of few rows as
in others: what equal weights lose to a rounding does not cancel, so it shows.

Of every 128 keys one scores ``gap`` and its value is 0, the others score 0 and their
values are 1: wherever the keys are shared out, the one is what weights refer to.
With n equal keys and m others the output is n e^-gap / (m + n e^-gap), and it is off,
relative to itself, by
  u = eps / 2    its own rounding,
  2^-11          the weights' to fp16: e^-13 2^7 is above 2^-14, so all are normal,
  n 2^-24        n additions of products of ones, each off by 2^-24 of the sum at most,
  2^-15          the rest in 32 bits: an exponent of at most 32 in a step of 2^-19 and
                 its factor by 3 roundings of 13 log2 e, so 2^-18 of a weight; the
                 exponential 2^-22, twice where a reference moves; the sum of weights
                 n / 64 + 16 additions a thread, 2^-18; the joining 2^-20.
The scores are exact: queries of ones, keys of one number that is not 0."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda

from .test_paged_attention_quant_gpu import BF16, F8, FP16, Case, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,heads", [(1, 1), (2, 4), (4, 4), (1, 10), (5, 4), (40, 1), (150, 2)])
def test_equal_weights_keep_their_bits(rows, heads, dtype):
    n = 2000
    c = Case([rows], [n], heads, 1, 64, dtype, seed=13)
    c.q[...] = 1.0
    c.k.view(torch.uint8).zero_()
    c.ks[:], c.vs[:] = 1.0, 2.0 ** -7
    c.v.view(torch.uint8)[...] = torch.tensor(128.0).to(F8).view(torch.uint8).item()
    for page, row in c.rows(0)[5::128]:
        c.set(c.k, (page, row, 0, 0), 1.0)
        c.v.view(torch.uint8)[page, row] = 0
    seen = n - rows + 1 + np.arange(rows)[:, None]  # keys that each token sees
    high = (seen - 6) // 128 + 1
    equal = seen - high
    tol = torch.finfo(dtype).eps / 2 + 2.0 ** -11 + n * 2.0 ** -24 + 2.0 ** -15
    for gap in np.linspace(2.0, 13.0, 150):
        c.scale = float(np.float32(gap))
        out, lse = c.run()
        others = equal * np.exp(-c.scale)
        want = (others / (high + others))[..., None]
        off = np.abs(_np(out) - want) / want
        assert off.max() <= tol, (gap, off.max(), tol)
        assert np.abs(_np(lse) - c.scale - np.log(high + others)).max() <= 2.0 ** -13
    assert kda.kda_device_status() == 0
