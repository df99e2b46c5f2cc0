"""Rotary positions: the handle that a serving program keeps, and the call of
include/kda.h on it.  Argument marshalling, and the frequencies of the
rotation, which are worked out once on the host."""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import torch

from . import _native
from .kv_cache import _DTYPES, _check_stream, _int32, _rows, _stream

LAYOUTS = ("half", "pairs")
_TWO_PI = Fraction(0x3243F6A8885A308D313198A2E0370734, 1 << 123)


def rope_frequencies(dim: int = 128, base: float = 10000.0, *, factor: float = 1.0, original_context: int = 0,
                     low: float = 1.0, high: float = 4.0) -> torch.Tensor:
    """Radians a position of the dim / 2 pairs of the first ``dim`` dimensions,
    f_i = base^(-2i / dim), float64 on the host.  For contexts ``factor`` times
    as long as those that a model was made for: f_i / factor; or, with
    ``original_context`` > 0, by how often a pair turns over that many tokens,
    r = original_context f_i / 2 pi: f_i where r >= high, f_i / factor where
    r <= low, and in between f_i (w + (1 - w) / factor), w = (r - low) / (high - low)."""
    if dim % 2 or not 2 <= dim <= 128:
        raise ValueError(f"dim must be even and in 2 .. 128 (got {dim}).")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor > 0):
        raise ValueError("base and factor must be positive and finite.")
    if original_context < 0 or not low < high:
        raise ValueError("original_context must be >= 0 and low < high.")
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    if not original_context:
        return f / factor
    w = ((original_context * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    return f * (w + (1 - w) / factor)


class Rope:
    """A rotation by ``frequencies`` [pairs] (radians a position, at most 64,
    a float64 tensor or a list, :func:`rope_frequencies`), of pairs (x_i,
    x_{i + pairs}) with the layout "half", (x_2i, x_{2i+1}) with "pairs"; the
    turned pairs times ``amplitude``."""

    def __init__(self, frequencies, *, layout: str = "half", amplitude: float = 1.0, device="cuda"):
        f = [float(x) for x in frequencies]
        if not 1 <= len(f) <= 64 or not all(map(math.isfinite, f)):
            raise ValueError("frequencies must be 1 to 64 finite numbers.")
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {LAYOUTS} (got {layout!r}).")
        if not math.isfinite(amplitude):
            raise ValueError("amplitude must be finite.")
        # a position's turns as a fraction of 2^64, in a signed tensor
        turns = [round(Fraction(x) / _TWO_PI * (1 << 64)) % (1 << 64) for x in f]
        self.turns = torch.tensor([x - (1 << 64) if x >> 63 else x for x in turns], dtype=torch.int64, device=device)
        if not self.turns.is_cuda:
            raise ValueError("a rotation lives on a CUDA device.")
        r = self._struct = _native.KdaRotation()
        r.turns, r.pairs, r.interleaved, r.amplitude = self.turns.data_ptr(), len(f), int(layout == "pairs"), amplitude
        self.dim, self.layout, self.amplitude = 2 * len(f), layout, amplitude
        self._index = self.turns.get_device()
        self._ref = ctypes.byref(r)


def _out(y, x, name, dtype, index):
    """(pointer, token stride, head stride) of the output y of x."""
    if y is not x and y.shape != x.shape:
        raise ValueError(f"{name}_out must have {name}'s shape.")
    return _rows(y, f"{name}_out", dtype, index)[2:]


def kda_rope(rope: Rope, q, k=None, *, positions=None, cu_seqlens=None, kv_lens=None, q_out=None, k_out=None, stream=None):
    """Turn q [T, Hq, 128] and k [T, Hkv, 128] (bf16 or fp16; k may be None) by
    the positions of their tokens: ``positions`` [T], or, from ``cu_seqlens``
    and ``kv_lens`` as :func:`kda_paged_attention` takes them, token i of the n
    of request b at kv_lens[b] - n + i (tokens of no request are left alone).
    Returns (q_out, k_out), new tensors unless given; ``q_out=q`` turns in
    place.  What the call makes belongs to ``stream``, as in
    :func:`kda_kv_extend`."""
    index = rope._index
    if stream is not None:
        _check_stream(stream, index)
        with torch.cuda.stream(stream):
            return kda_rope(rope, q, k, positions=positions, cu_seqlens=cu_seqlens, kv_lens=kv_lens, q_out=q_out, k_out=k_out)
    handle, dtype = _stream(None, index), q.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"q must be torch.bfloat16 or torch.float16 (got {dtype}).")
    t, hq, qp, qt, qh = _rows(q, "q", dtype, index)
    if q_out is None:
        q_out = torch.empty((t, hq, 128), dtype=dtype, device=q.device)
        out = q_out.data_ptr(), hq * 128, 128
    else:
        out = _out(q_out, q, "q", dtype, index)
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k.")
        hk, kp, kt, kh, k_args = 0, None, 0, 0, (None, 0, 0)
    else:
        tk, hk, kp, kt, kh = _rows(k, "k", dtype, index)
        if tk != t:
            raise ValueError("q and k must have the same number of tokens.")
        if k_out is None:
            k_out = torch.empty((t, hk, 128), dtype=dtype, device=k.device)
            k_args = k_out.data_ptr(), hk * 128, 128
        else:
            k_args = _out(k_out, k, "k", dtype, index)
    n = 0
    if positions is not None:
        if cu_seqlens is not None or kv_lens is not None:
            raise ValueError("positions, or cu_seqlens and kv_lens, not both.")
        where = (_int32(positions, "positions", index, t), None, None)
    elif cu_seqlens is None or kv_lens is None:
        raise ValueError("positions, or cu_seqlens and kv_lens, are needed.")
    else:
        n = kv_lens.numel()
        where = (None, _int32(cu_seqlens, "cu_seqlens", index, n + 1), _int32(kv_lens, "kv_lens", index))
    rc = _native.lib().kda_rope(rope._ref, _DTYPES[dtype], qp, qt, qh, hq, *out, kp, kt, kh, hk, *k_args, t, *where, n, handle)
    if rc:
        _native.check(rc)
    return q_out, k_out
