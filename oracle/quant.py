"""The 8-bit key/value cache and rotary positions written out, in numpy fp64."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16
TOP = 448.0
LEAST, MOST = -48, 48


def round_e4m3(x):
    """To the nearest of the numbers with 4 significant bits on a grid of 2^-9,
    ties to even; past 448, infinities too, 448; NaN stays."""
    x = np.clip(np.asarray(x, dtype=np.float64), -2 * TOP, 2 * TOP)
    _, e = np.frexp(np.where(np.isnan(x) | (x == 0), 1.0, np.abs(x)))  # x = m 2^e, 1/2 <= m < 1
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.clip(np.rint(x / step) * step, -TOP, TOP)


def exponent(m):
    """Least e in [LEAST, MOST] with m <= 448 2^e (MOST where none is)."""
    return next((e for e in range(LEAST, MOST) if m <= TOP * 2.0 ** e), MOST)


def append(cache, scales, x, slots):
    """Numbers ``cache`` [pages, page, H, 128] and ``scales`` [pages, H, page /
    16] (fp64 arrays), updated in place with x [T, H, 128] at ``slots``, whose
    blocks' tokens stand side by side."""
    page = cache.shape[1]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        end = t + 1
        while end < len(slots) and slots[end] == slots[t] + end - t and slots[end] % BLOCK:
            end += 1
        pg, row = divmod(slots[t], page)
        b, r0 = divmod(row, BLOCK)
        for h in range(x.shape[1]):
            new = x[t:end, h]
            scale = 2.0 ** exponent(np.max(np.abs(new), initial=0.0, where=np.isfinite(new)))
            if r0 and scales[pg, h, b] >= scale:
                scale = scales[pg, h, b]
            elif r0:
                cache[pg, row - r0:row, h] = round_e4m3(cache[pg, row - r0:row, h] * (scales[pg, h, b] / scale))
            scales[pg, h, b] = scale
            cache[pg, row:row + end - t, h] = round_e4m3(new / scale)
        t = end


def values(cache, scales):
    """What the cache stands for: [pages, page, H, 128]."""
    return cache * np.repeat(scales, BLOCK, 2).transpose(0, 2, 1)[..., None]


def rope(x, positions, frequencies, layout="half", amplitude=1.0):
    """x [T, H, 128] turned by positions [T]."""
    n = len(frequencies)
    y = np.array(x, dtype=np.float64)
    for i, f in enumerate(frequencies):
        a, b = (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + n)
        c = np.array([math.cos(p * f) for p in positions])[:, None]
        s = np.array([math.sin(p * f) for p in positions])[:, None]
        y[..., a], y[..., b] = amplitude * (x[..., a] * c - x[..., b] * s), amplitude * (x[..., b] * c + x[..., a] * s)
    return y
