"""Refusals of the 8-bit cache's and the rotation's entry points, without a GPU:
each broken rule of include/kda.h fails before any launch.  Pointers are fake,
aligned addresses that are never read."""
from __future__ import annotations

import ctypes

import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from linear_attention_serving_fwd_gb300 import _native

INVALID, DTYPE = 1, 2
FAKE = 0x10000


def _msg():
    return _native.lib().kda_last_error().decode()


def _cache(**over):
    c = _native.KdaKvQuantCache()
    c.k = c.v = c.k_scale = c.v_scale = FAKE
    c.k_stride_page = c.v_stride_page = 16 * 2 * 128
    c.k_stride_tok = c.v_stride_tok = 2 * 128
    c.k_stride_head = c.v_stride_head = 128
    c.dtype, c.n_pages, c.page_size, c.hkv = 0, 32, 16, 2
    for k, v in over.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def _append(cache, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, slots=FAKE, t=4):
    return _native.lib().kda_kv_append_quant(cache, k, kt, kh, v, vt, 128, slots, t, None)


def _read(cache, slots=FAKE, t=4, k=FAKE, v=FAKE):
    return _native.lib().kda_kv_read_quant(cache, slots, t, k, v, None)


def _attend(cache, q=FAKE, qt=512, qh=128, hq=4, t=4, out=FAKE, cu=FAKE, lens=FAKE, table=FAKE, stride=8, cols=8, n=2,
            scale=0.1, window=0, sinks=0, ws=FAKE, ws_bytes=1 << 40):
    return _native.lib().kda_paged_attention_quant(cache, q, qt, qh, hq, t, out, None, cu, lens, table, stride, cols, n,
                                                   scale, window, sinks, ws, ws_bytes, None)


@pytest.mark.parametrize("over,code,text", [
    (dict(dtype=2), DTYPE, "bfloat16 or float16"), (dict(page_size=48), INVALID, "page_size"),
    (dict(n_pages=0), INVALID, "n_pages"), (dict(n_pages=1 << 28), INVALID, "2^31"), (dict(hkv=0), INVALID, "hkv"),
    (dict(k=None), INVALID, "NULL"), (dict(v_scale=None), INVALID, "NULL"), (dict(v=FAKE + 8), INVALID, "16-byte aligned"),
    (dict(k_scale=FAKE + 2), INVALID, "4-byte aligned"), (dict(k_stride_tok=264), INVALID, "multiples of 16"),
    (dict(v_stride_head=0), INVALID, "multiples of 16"), (dict(v_stride_page=-4096), INVALID, "multiples of 16"),
])
def test_cache(over, code, text):
    for call in (_append, _read, _attend):
        assert call(_cache(**over)) == code and text in _msg()
    assert _append(None) == _read(None) == _attend(None) == INVALID


@pytest.mark.parametrize("over,text", [
    (dict(k=None), "k must not be NULL"), (dict(k=FAKE + 2), "aligned"), (dict(kt=129), "multiples of 8"),
    (dict(kh=-128), "multiples of 8"), (dict(v=None), "v must not be NULL"), (dict(vt=-8), "v strides"),
    (dict(slots=None), "slot_map"), (dict(t=-1), "t_total"),
])
def test_append(over, text):
    assert _append(_cache(), **over) == INVALID and text in _msg()


@pytest.mark.parametrize("over,text", [
    (dict(slots=None), "slot_map"), (dict(t=-1), "t_total"), (dict(k=None), "k and v"), (dict(v=FAKE + 8), "aligned"),
])
def test_read(over, text):
    assert _read(_cache(), **over) == INVALID and text in _msg()
    c = _native.KdaKvCache()
    c.k = c.v = FAKE
    c.k_stride_page = c.v_stride_page = c.k_stride_tok = c.v_stride_tok = c.k_stride_head = c.v_stride_head = 4096
    c.n_pages, c.page_size, c.hkv = 32, 16, 2
    a = {**dict(slots=FAKE, t=4, k=FAKE, v=FAKE), **over}
    assert _native.lib().kda_kv_read(ctypes.byref(c), a["slots"], a["t"], a["k"], a["v"], None) == INVALID and text in _msg()


@pytest.mark.parametrize("over,text", [
    (dict(hq=3), "multiple of key heads"), (dict(hq=0), "multiple of key heads"), (dict(hq=258), "at most 128"),
    (dict(t=-1), ">= 0"), (dict(n=-1), ">= 0"), (dict(scale=0.0), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(window=-1), "window"), (dict(sinks=-1), "sinks"), (dict(q=None), "q must not be NULL"),
    (dict(q=FAKE + 4), "aligned"), (dict(qt=4), "multiples of 8"), (dict(qt=8), "overlap"), (dict(out=None), "out must not"),
    (dict(out=FAKE + 16), "out must be 32"), (dict(cu=None), "cu_seqlens"), (dict(lens=None), "kv_lens"),
    (dict(table=None), "block_table"), (dict(cols=0), "column"), (dict(stride=7), "table_stride"),
    (dict(cols=(1 << 27), stride=1 << 27), "2^31"), (dict(ws=None), "workspace needs"), (dict(ws_bytes=64), "workspace needs"),
    (dict(ws=FAKE + 8), "workspace must be"),
])
def test_attention(over, text):
    assert _attend(_cache(), **over) == INVALID and text in _msg()


def test_the_workspace_grows_with_the_queries():
    size = _native.lib().kda_paged_attention_quant_workspace_bytes
    wide = _native.lib().kda_paged_attention_workspace_bytes()
    assert size(0, 0) >= wide and size(1000, 32) > size(1000, 16) > size(10, 16) and size(-1, 4) == size(0, 4)
    assert _attend(_cache(), t=64, ws_bytes=size(63, 4)) == INVALID and "workspace needs" in _msg()


def _rope(pairs=64, interleaved=0, amplitude=1.0, turns=FAKE, dtype=0, q=FAKE, qt=512, qh=128, hq=4, q_out=FAKE + (1 << 20),
          qot=512, qoh=128, k=FAKE, hk=2, k_out=FAKE + (1 << 20), t=4, positions=None, cu=FAKE, lens=FAKE, n=2):
    r = _native.KdaRotation()
    r.turns, r.pairs, r.interleaved, r.amplitude = turns, pairs, interleaved, amplitude
    return _native.lib().kda_rope(ctypes.byref(r), dtype, q, qt, qh, hq, q_out, qot, qoh, k, 256, 128, hk, k_out, 256, 128, t,
                                  positions, cu, lens, n, None)


@pytest.mark.parametrize("over,code,text", [
    (dict(pairs=0), INVALID, "pairs"), (dict(pairs=65), INVALID, "pairs"), (dict(interleaved=2), INVALID, "interleaved"),
    (dict(amplitude=float("inf")), INVALID, "amplitude"), (dict(turns=None), INVALID, "turns"),
    (dict(turns=FAKE + 4), INVALID, "8-byte"), (dict(dtype=2), DTYPE, "bfloat16 or float16"), (dict(hq=-1), INVALID, ">= 0"),
    (dict(hk=-1), INVALID, ">= 0"), (dict(t=-1), INVALID, ">= 0"), (dict(n=-1), INVALID, ">= 0"),
    (dict(q=None), INVALID, "q must not be NULL"), (dict(q_out=None), INVALID, "q_out must not be NULL"),
    (dict(k=FAKE + 8), INVALID, "k must be 16-byte"), (dict(k_out=None), INVALID, "k_out must not"),
    (dict(qt=8), INVALID, "q rows must not overlap"), (dict(qoh=64), INVALID, "q_out rows must not overlap"),
    (dict(qh=132), INVALID, "multiples of 8"), (dict(q_out=FAKE, qot=1024), INVALID, "in place"),
    (dict(cu=None), INVALID, "positions"), (dict(lens=None), INVALID, "positions"),
])
def test_rope(over, code, text):
    assert _rope(**over) == code and text in _msg()


def test_nothing_to_do():
    assert _append(_cache(), t=0, k=None) == 0
    assert _read(_cache(), t=0, k=None) == 0
    assert _attend(_cache(), t=0, q=None) == 0
    assert _attend(_cache(), n=0, cu=None) == 0
    assert _rope(t=0, q=None) == 0 and _rope(hq=0, hk=0, q=None) == 0 and _rope(n=0, cu=None) == 0
    assert _native.lib().kda_rope(None, 0, FAKE, 512, 128, 4, FAKE, 512, 128, None, 0, 0, 0, None, 0, 0, 4, FAKE, None, None, 0,
                                  None) == INVALID


def test_python_refusals():
    x = torch.zeros(4, 16, 2, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(4, 2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        kda.KvCache(x, x, s, s, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        kda.KvCache(x, x.view(torch.uint8), s, s, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        kda.KvCache(x.view(torch.float8_e5m2), x.view(torch.float8_e5m2), s, s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.Rope([1.0], device="cpu")
    for bad in ([], [1.0] * 65, [float("nan")]):
        with pytest.raises(ValueError, match="frequencies"):
            kda.Rope(bad, device="cpu")
    with pytest.raises(ValueError, match="layout"):
        kda.Rope([1.0], layout="both", device="cpu")
    with pytest.raises(ValueError, match="amplitude"):
        kda.Rope([1.0], amplitude=float("inf"), device="cpu")
