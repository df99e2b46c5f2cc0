"""The paged key/value cache of softmax-attention layers: the handles that a
serving program keeps, and the calls of include/kda.h on them.

A step of such a program is: :func:`kda_kv_extend` takes pages for its new
tokens, each layer writes its keys and values with :func:`kda_kv_append` and
runs :func:`kda_paged_attention`; :func:`kda_kv_truncate` hands the pages of
rejected drafts and finished requests back.  Argument marshalling only.  A
call's tensors and its stream are on its handle's device, which is the current
one; what a call makes for itself or returns is made on its stream, so that a
workspace is zeroed there first and memory is reused in its order.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _native

D = 128
_DTYPES = {torch.bfloat16: _native.KDA_DTYPE_BF16, torch.float16: _native.KDA_DTYPE_FP16}


# The current stream's handle without the object around it: a decode step makes
# a few of these calls per layer, and the object costs more than a launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


# The current device's number, without the set-up checks around it: a handle's
# tensors are there already.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream, index):
    """The handle of the call's stream.  The launch, the error word and the
    workspace's size are the current device's: it has to be the handles'."""
    if _current_device() != index:
        raise ValueError(f"the current device must be the handles' device cuda:{index}.")
    if stream is None:
        return _raw_stream(index)
    _check_stream(stream, index)
    return stream.cuda_stream


def _check_stream(stream, index):
    if stream.device.index != index:
        raise ValueError(f"stream must be of cuda:{index} (got {stream.device}).")


def _refuse(t, name, index, kind):
    """The error for a tensor that is not ``kind``, or not on cuda:``index``."""
    if t.is_cuda and t.get_device() != index:
        return ValueError(f"{name} must be on cuda:{index} with the handles (got {t.device}).")
    return TypeError(f"{name} must be {kind} (got {t.dtype} on {t.device}).")


def _int32(t, name, index, numel=None):
    if t.dtype != torch.int32 or t.get_device() != index or not t.is_contiguous():
        raise _refuse(t, name, index, "a contiguous int32 CUDA tensor")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} entries (got {t.numel()}).")
    return t.data_ptr()


def _table(t, n_req, index):
    """(pointer, row stride, columns)"""
    if t.dtype != torch.int32 or t.get_device() != index:
        raise _refuse(t, "block_table", index, "an int32 CUDA tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != n_req or (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"block_table must be [{n_req}, columns] with contiguous rows (got {tuple(shape)}).")
    return t.data_ptr(), stride[0], shape[1]


def _rows(t, name, dtype, index, heads=None):
    """(tokens, heads, pointer, token stride, head stride) of [T, H, 128] in the
    cache's type; a size-1 dimension's stride is free."""
    if t.dtype != dtype or t.get_device() != index:
        raise _refuse(t, name, index, f"a CUDA tensor of the cache's dtype {dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != D or stride[2] != 1 or (heads is not None and shape[1] != heads):
        want = "H" if heads is None else heads
        raise ValueError(f"{name} must be [T, {want}, 128] with a contiguous last dimension (got {tuple(shape)}).")
    n, h, _ = shape
    return n, h, t.data_ptr(), stride[0] if n > 1 else 0, stride[1] if h > 1 else 0


class KvPages:
    """Who owns which page: ``kv_lens`` [n_req], ``block_table`` [n_req,
    columns], the stack ``free_pages`` [n_pages] and its height ``free_count``
    [1], all int32 CUDA tensors that :func:`kda_kv_extend` and
    :func:`kda_kv_truncate` update in place.  :meth:`empty` makes a pool in
    which every page is free."""

    def __init__(self, kv_lens, block_table, free_pages, free_count, page_size: int):
        n = kv_lens.numel()
        g = self._struct = _native.KdaKvPages()
        index = self._index = max(0, kv_lens.get_device())
        g.kv_lens = _int32(kv_lens, "kv_lens", index)
        g.block_table, g.table_stride, g.table_cols = _table(block_table, n, index)
        g.free_pages, g.free_count = _int32(free_pages, "free_pages", index), _int32(free_count, "free_count", index, 1)
        g.n_req, g.n_pages, g.page_size = n, free_pages.numel(), page_size
        self.n_req, self.device = n, kv_lens.device
        self.kv_lens, self.block_table = kv_lens, block_table
        self.free_pages, self.free_count, self.page_size = free_pages, free_count, page_size
        self._ref = ctypes.byref(g)

    @classmethod
    def empty(cls, n_req: int, columns: int, n_pages: int, page_size: int, device="cuda") -> "KvPages":
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros(n_req, **i32), torch.full((n_req, columns), -1, **i32),
                   torch.arange(n_pages - 1, -1, -1, **i32), torch.full((1,), n_pages, **i32), page_size)


class KvCache:
    """The pages' storage: ``k`` and ``v`` as [n_pages, page_size, Hkv, 128]
    CUDA tensors of any strides that are multiples of 8 elements with a
    contiguous last dimension (a permuted view of head-major pages, halves of
    one tensor), bf16 or fp16."""

    def __init__(self, k, v):
        if k.dtype not in _DTYPES or v.dtype != k.dtype:
            raise TypeError("the cache must be torch.bfloat16 or torch.float16, k and v alike.")
        if k.dim() != 4 or k.shape != v.shape or k.shape[3] != D or k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v must be [n_pages, page_size, Hkv, 128] alike with a contiguous last dimension.")
        if not k.is_cuda or v.device != k.device:
            raise ValueError("k and v must be CUDA tensors on one device.")
        c = self._struct = _native.KdaKvCache()
        for name, t in (("k", k), ("v", v)):
            setattr(c, name, t.data_ptr())
            for dim, what in ((0, "page"), (1, "tok"), (2, "head")):
                # the stride of a dimension of size 1 is never used
                setattr(c, f"{name}_stride_{what}", t.stride(dim) if t.shape[dim] > 1 else D)
        c.dtype = _DTYPES[k.dtype]
        c.n_pages, c.page_size, c.hkv = k.shape[:3]
        self.k, self.v, self.dtype, self.n_kv_heads = k, v, k.dtype, k.shape[2]
        self._index = k.get_device()
        self._ref = ctypes.byref(c)


def kda_kv_extend(pages: KvPages, new_lens, max_tokens: int, *, cu_seqlens=None, slot_map=None, step_lens=None,
                  stream=None):
    """Take the pages for ``new_lens`` [n_req] new tokens (int32, CUDA), at
    most ``max_tokens`` in all.  Updates ``pages``; returns (cu_seqlens
    [n_req + 1], slot_map [max_tokens], step_lens [n_req]), int32: the packed
    layout, each token's slot (-1 where its request found no pages), and the
    lengths that attention takes (0 where the request was not admitted).  What
    the call makes belongs to ``stream`` where one is given: another stream that
    uses it waits for that one, and records itself on the tensor."""
    index, n = pages._index, pages.n_req
    if stream is not None:
        _check_stream(stream, index)
        with torch.cuda.stream(stream):
            return kda_kv_extend(pages, new_lens, max_tokens, cu_seqlens=cu_seqlens, slot_map=slot_map, step_lens=step_lens)
    handle, new = _stream(None, index), _int32(new_lens, "new_lens", index, n)
    if cu_seqlens is None:
        cu_seqlens = torch.empty(n + 1, dtype=torch.int32, device=pages.device)
    if slot_map is None:
        slot_map = torch.empty(max_tokens, dtype=torch.int32, device=pages.device)
    if step_lens is None:
        step_lens = torch.empty(n, dtype=torch.int32, device=pages.device)
    rc = _native.lib().kda_kv_extend(
        pages._ref, new, _int32(cu_seqlens, "cu_seqlens", index, n + 1), _int32(slot_map, "slot_map", index, max_tokens),
        max_tokens, _int32(step_lens, "step_lens", index, n), handle)
    if rc:
        _native.check(rc)
    return cu_seqlens, slot_map, step_lens


def kda_kv_truncate(pages: KvPages, keep_lens, *, stream=None) -> None:
    """Keep the first ``keep_lens`` [n_req] tokens of each request (int32,
    CUDA) and hand the pages past them back.  A negative table entry, a page
    that the caller has handed back itself, is passed over."""
    index = pages._index
    rc = _native.lib().kda_kv_truncate(pages._ref, _int32(keep_lens, "keep_lens", index, pages.n_req), _stream(stream, index))
    if rc:
        _native.check(rc)


def kda_kv_append(cache: KvCache, k, v, slot_map, *, stream=None) -> None:
    """Write k and v [T, Hkv, 128] to the slots ``slot_map`` [T] (int32, -1
    skips the token)."""
    index = cache._index
    t, _, kp, kt, kh = _rows(k, "k", cache.dtype, index, cache.n_kv_heads)
    tv, _, vp, vt, vh = _rows(v, "v", cache.dtype, index, cache.n_kv_heads)
    if tv != t:
        raise ValueError("k and v must have the same number of tokens.")
    rc = _native.lib().kda_kv_append(cache._ref, kp, kt, kh, vp, vt, vh, _int32(slot_map, "slot_map", index, t), t,
                                     _stream(stream, index))
    if rc:
        _native.check(rc)


def paged_attention_workspace(device=None) -> torch.Tensor:
    """A workspace for :func:`kda_paged_attention`.  One serves any sequence
    of calls on one stream; calls that overlap need their own."""
    device = "cuda" if device is None else device
    with torch.cuda.device(device):  # the size goes by the current device
        n = int(_native.lib().kda_paged_attention_workspace_bytes())
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kda_paged_attention(cache: KvCache, q, cu_seqlens, kv_lens, block_table, *, scale: Optional[float] = None,
                        window: int = 0, sinks: int = 0, out=None, lse=None, return_lse: bool = False,
                        workspace=None, stream=None):
    """Causal attention of packed tokens q [T, Hq, 128] over the paged cache,
    which holds them already: request b owns tokens cu_seqlens[b] ..
    cu_seqlens[b+1]-1, the last of its kv_lens[b] cached ones.  With
    ``window`` > 0 a token sees the last ``window`` positions, its own among
    them, and the first ``sinks``.  Returns (out [T, Hq, 128], lse fp32
    [T, Hq] or None).  ``workspace``: :func:`paged_attention_workspace`, made
    for the call when not given.  What the call makes belongs to ``stream``, as
    in :func:`kda_kv_extend`."""
    index = cache._index
    if stream is not None:
        _check_stream(stream, index)
        with torch.cuda.stream(stream):
            return kda_paged_attention(cache, q, cu_seqlens, kv_lens, block_table, scale=scale, window=window, sinks=sinks,
                                       out=out, lse=lse, return_lse=return_lse, workspace=workspace)
    handle = _stream(None, index)
    t, hq, qp, qt, qh = _rows(q, "q", cache.dtype, index)
    n = kv_lens.numel()
    if out is None:
        out = torch.empty((t, hq, D), dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.get_device() != index:
        raise ValueError(f"out must be a contiguous tensor of q's shape and dtype on cuda:{index}.")
    if lse is None:
        lse = torch.empty((t, hq), dtype=torch.float32, device=q.device) if return_lse else None
    elif tuple(lse.shape) != (t, hq) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.get_device() != index:
        raise ValueError(f"lse must be a contiguous float32 tensor [T, Hq] on cuda:{index}.")
    if workspace is None:
        workspace = paged_attention_workspace(q.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{index}.")
    table, table_stride, cols = _table(block_table, n, index)
    rc = _native.lib().kda_paged_attention(
        cache._ref, qp, qt, qh, hq, t, out.data_ptr(), None if lse is None else lse.data_ptr(),
        _int32(cu_seqlens, "cu_seqlens", index, n + 1), _int32(kv_lens, "kv_lens", index), table, table_stride, cols, n,
        D ** -0.5 if scale is None else scale, window, sinks, workspace.data_ptr(), workspace.numel(), handle)
    if rc:
        _native.check(rc)
    return out, lse
