"""Narrow blocks over the 8-bit cache take a weight as three e5m2 numbers, the upper
bytes of fp16 ones, each remainder 16 times larger: written out for every fp16
number up to 32768, the sum is that number, and no step on the way is inexact or overflows."""
from __future__ import annotations

import numpy as np


def test_three_parts_are_the_weight():
    bits = np.arange(np.float16(32768).view(np.uint16) + 1, dtype=np.uint16)
    weight = bits.view(np.float16).astype(np.float64)
    total, left = np.zeros_like(weight), weight
    for part in range(3):
        h = left.astype(np.float16)
        assert (h.astype(np.float64) == left).all()
        up = h.view(np.uint16).astype(np.uint32) + (0x80 if part < 2 else 0)
        assert ((up ^ h.view(np.uint16)) < 0x8000).all()  # the sign stays
        top = (up & 0xff00).astype(np.uint16).view(np.float16).astype(np.float64)
        assert np.isfinite(top).all()
        total += top / 16.0 ** part
        left = (left - top) * 16
    assert (total == weight).all()
