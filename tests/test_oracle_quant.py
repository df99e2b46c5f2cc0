"""Pins of the 8-bit cache's and the rotation's oracle: e4m3 against torch's
own conversion, scales at their borders by hand, rotations against quarter
turns, composition and complex numbers."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from oracle import quant


def _all_numbers():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    return np.unique(codes[np.isfinite(codes)])


def test_rounding_is_torchs():
    n = _all_numbers()
    assert n.max() == 448 and (quant.round_e4m3(n) == n).all()
    mid = (n[1:] + n[:-1]) / 2
    x = np.concatenate([mid, mid * (1 + 1e-6), mid * (1 - 1e-6), np.random.default_rng(0).normal(0, 50, 10000)])
    want = torch.tensor(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert (quant.round_e4m3(x.astype(np.float32)) == want).all()


def test_rounding_past_the_largest():
    got = quant.round_e4m3([448.1, 464, 1e30, np.inf, -np.inf, -449])
    assert got.tolist() == [448, 448, 448, 448, -448, -448] and np.isnan(quant.round_e4m3(np.nan))


@pytest.mark.parametrize("m,e", [(448, 0), (448.001, 1), (224, -1), (224.01, 0), (0, -48), (1e-30, -48), (1e30, 48),
                                 (1.75 * 2.0 ** -10, -18), (1.751 * 2.0 ** -10, -17), (448 * 2.0 ** 48, 48)])
def test_exponents(m, e):
    assert quant.exponent(m) == e


def test_a_block_grows():
    cache, scales = np.zeros((1, 16, 1, 128)), np.ones((1, 1, 1))
    quant.append(cache, scales, np.full((2, 1, 128), 3.0), [0, 1])
    assert scales[0, 0, 0] == 2.0 ** -7 and (cache[0, :2] == 384).all()
    quant.append(cache, scales, np.full((1, 1, 128), 1.0), [2])  # the larger scale stays
    assert scales[0, 0, 0] == 2.0 ** -7 and (cache[0, 2] == 128).all()
    quant.append(cache, scales, np.full((1, 1, 128), 3000.0), [3])
    assert scales[0, 0, 0] == 8 and (cache[0, :2] == 0.375).all() and (cache[0, 2] == 0.125).all()
    assert np.array_equal(quant.values(cache, scales)[0, :4, 0, 0], [3, 3, 1, 384 * 8])
    quant.append(cache, scales, np.full((1, 1, 128), 1.0), [0])  # a new tenant of the block
    assert scales[0, 0, 0] == 2.0 ** -8


def test_rotation_by_quarter_turns():
    x = np.random.default_rng(1).normal(size=(4, 2, 128))
    for layout in ("half", "pairs"):
        y = quant.rope(x, [0, 1, 2, 3], [math.pi / 2] * 64, layout)
        a, b = (x[..., :64], x[..., 64:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
        c, d = (y[..., :64], y[..., 64:]) if layout == "half" else (y[..., 0::2], y[..., 1::2])
        for t, (u, v) in enumerate([(a, b), (-b, a), (-a, -b), (b, -a)]):
            np.testing.assert_allclose(c[t], u[t], atol=1e-12)
            np.testing.assert_allclose(d[t], v[t], atol=1e-12)


def test_products_depend_on_the_distance_alone():
    r = np.random.default_rng(2)
    q, k = r.normal(size=(1, 1, 128)), r.normal(size=(1, 1, 128))
    f = kda.rope_frequencies(96, 1e4).tolist()
    for layout in ("half", "pairs"):
        dots = [float((quant.rope(q, [p + 5], f, layout) * quant.rope(k, [p], f, layout)).sum()) for p in (0, 7, 1000)]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-10)
        y = quant.rope(q, [3], f, layout)
        assert (y[..., 96:] == q[..., 96:]).all() and abs(np.linalg.norm(y) - np.linalg.norm(q)) < 1e-12


def test_frequencies():
    f = kda.rope_frequencies(128, 10000.0)
    assert f[0] == 1 and abs(f[32] - 0.01) < 1e-15 and f.dtype == torch.float64
    assert torch.equal(kda.rope_frequencies(64, 1e6, factor=8.0), kda.rope_frequencies(64, 1e6) / 8)
    g = kda.rope_frequencies(128, 5e5, factor=8.0, original_context=8192)
    f = kda.rope_frequencies(128, 5e5)
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 4], f[turns >= 4]) and torch.allclose(g[turns <= 1], f[turns <= 1] / 8)
    between = (turns > 1) & (turns < 4)
    w = (turns[between] - 1) / 3
    assert between.any() and torch.allclose(g[between], f[between] * (w + (1 - w) / 8))
    for bad in (dict(dim=3), dict(dim=0), dict(dim=130), dict(base=0.0), dict(factor=-1.0), dict(original_context=-1),
                dict(low=4.0, high=4.0), dict(base=float("nan"))):
        with pytest.raises(ValueError):
            kda.rope_frequencies(**{"dim": 64, **bad})
