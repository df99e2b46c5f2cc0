"""Refusals of the paged cache's entry points, without a GPU: each broken rule
of include/kda.h fails before any launch.  Pointers are fake, aligned
addresses that are never read."""
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


def _pages(**over):
    g = _native.KdaKvPages()
    g.kv_lens = g.block_table = g.free_pages = g.free_count = FAKE
    g.table_stride, g.n_req, g.table_cols, g.n_pages, g.page_size = 8, 4, 8, 32, 16
    for k, v in over.items():
        setattr(g, k, v)
    return ctypes.byref(g)


def _cache(**over):
    c = _native.KdaKvCache()
    c.k = c.v = FAKE
    c.k_stride_page = c.v_stride_page = 16 * 2 * 128
    c.k_stride_tok = c.v_stride_tok = 2 * 128
    c.k_stride_head = c.v_stride_head = 128
    c.dtype, c.n_pages, c.page_size, c.hkv = 0, 32, 16, 2
    for k, v in over.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def _extend(pages, new=FAKE, cu=FAKE, slots=FAKE, most=64, step=FAKE):
    return _native.lib().kda_kv_extend(pages, new, cu, slots, most, step, None)


PAGES = [
    (dict(page_size=24), "page_size"), (dict(page_size=8), "page_size"), (dict(page_size=512), "page_size"),
    (dict(n_pages=0), "n_pages"), (dict(n_pages=1 << 28), "2^31"), (dict(n_req=-1), "n_req"),
    (dict(kv_lens=None), "kv_lens"), (dict(block_table=None), "block_table"), (dict(free_pages=None), "free_pages"),
    (dict(free_count=None), "free_count"), (dict(table_cols=0), "column"), (dict(table_stride=7), "table_stride"),
    (dict(table_cols=1 << 28, table_stride=1 << 28), "2^31"),
]


@pytest.mark.parametrize("over,text", PAGES)
def test_pages(over, text):
    assert _extend(_pages(**over)) == INVALID and text in _msg()
    assert _native.lib().kda_kv_truncate(_pages(**over), FAKE, None) == INVALID and text in _msg()


def test_extend_and_truncate_pointers():
    assert _extend(None) == INVALID
    assert _extend(_pages(), most=-1) == INVALID and "max_tokens" in _msg()
    assert _extend(_pages(), new=None) == INVALID and "new_lens" in _msg()
    assert _extend(_pages(), cu=None) == INVALID and "cu_seqlens" in _msg()
    assert _extend(_pages(), slots=None) == INVALID and "slot_map" in _msg()
    assert _extend(_pages(), step=None) == INVALID and "step_lens" in _msg()
    assert _native.lib().kda_kv_truncate(_pages(), None, None) == INVALID and "keep_lens" in _msg()


CACHE = [
    (dict(dtype=2), DTYPE, "bfloat16 or float16"), (dict(page_size=48), INVALID, "page_size"),
    (dict(n_pages=0), INVALID, "n_pages"), (dict(hkv=0), INVALID, "hkv"), (dict(k=None), INVALID, "NULL"),
    (dict(v=FAKE + 8), INVALID, "16-byte aligned"), (dict(k_stride_tok=260), INVALID, "multiples of 8"),
    (dict(v_stride_head=0), INVALID, "multiples of 8"), (dict(v_stride_page=-4096), INVALID, "multiples of 8"),
]


def _append(cache, k=FAKE, kt=256, kh=128, v=FAKE, slots=FAKE, t=4):
    return _native.lib().kda_kv_append(cache, k, kt, kh, v, 256, 128, slots, t, None)


def _attend(cache, q=FAKE, qt=512, qh=128, hq=4, t=4, out=FAKE, cu=FAKE, lens=FAKE, table=FAKE, stride=8, cols=8, n=2,
            scale=0.1, window=0, sinks=0, ws=FAKE, ws_bytes=1 << 40):
    return _native.lib().kda_paged_attention(cache, q, qt, qh, hq, t, out, None, cu, lens, table, stride, cols, n, scale,
                                             window, sinks, ws, ws_bytes, None)


@pytest.mark.parametrize("over,code,text", CACHE)
def test_cache(over, code, text):
    assert _append(_cache(**over)) == code and text in _msg()
    assert _attend(_cache(**over)) == code and text in _msg()


@pytest.mark.parametrize("over,text", [
    (dict(k=None), "k must not be NULL"), (dict(k=FAKE + 2), "aligned"), (dict(kt=129), "multiples of 8"),
    (dict(kh=-128), "multiples of 8"), (dict(v=None), "v must not be NULL"), (dict(slots=None), "slot_map"),
    (dict(t=-1), "t_total"),
])
def test_append(over, text):
    assert _append(_cache(), **over) == INVALID and text in _msg()


@pytest.mark.parametrize("over,text", [
    (dict(hq=3), "multiple of key heads"), (dict(hq=0), "multiple of key heads"), (dict(hq=258), "at most 128"),
    (dict(t=-1), ">= 0"), (dict(n=-1), ">= 0"), (dict(scale=0.0), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(scale=-1.0), "scale"), (dict(window=-1), "window"),
    (dict(sinks=-1), "sinks"), (dict(q=None), "q must not be NULL"), (dict(q=FAKE + 4), "aligned"),
    (dict(qt=4), "multiples of 8"), (dict(out=None), "out must not"), (dict(out=FAKE + 16), "out must be 32"),
    (dict(cu=None), "cu_seqlens"), (dict(lens=None), "kv_lens"), (dict(table=None), "block_table"),
    (dict(cols=0), "column"), (dict(stride=7), "table_stride"), (dict(cols=(1 << 27), stride=1 << 27), "2^31"),
    (dict(ws=None), "workspace needs"), (dict(ws_bytes=64), "workspace needs"), (dict(ws=FAKE + 8), "workspace must be"),
])
def test_attention(over, text):
    assert _attend(_cache(), **over) == INVALID and text in _msg()


def test_nothing_to_do():
    assert _append(_cache(), t=0, k=None) == 0
    assert _attend(_cache(), t=0, q=None) == 0
    assert _attend(_cache(), n=0, cu=None) == 0
    assert _native.lib().kda_kv_truncate(_pages(n_req=0, kv_lens=None, block_table=None), None, None) == 0


def test_host_tensors_are_refused():
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        kda.KvPages(i32, torch.zeros(4, 8, dtype=torch.int32), i32, i32[:1], 16)
    with pytest.raises(TypeError, match="CUDA"):
        kda.KvPages.empty(4, 8, 32, 16, device="cpu")
    x = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.KvCache(x, x)
    with pytest.raises(TypeError):
        kda.KvCache(x.float(), x.float())
    with pytest.raises(TypeError):
        kda.KvCache(x, x.half())
    with pytest.raises(ValueError, match="128"):
        kda.KvCache(x[..., :64], x[..., :64])
    with pytest.raises(ValueError, match="alike"):
        kda.KvCache(x, x[:2])
