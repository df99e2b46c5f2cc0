"""The Python side of the paged cache's calls, without a GPU: CPU tensors that
claim to be CUDA ones, and a library that notes its calls."""
from __future__ import annotations

import contextlib
import types

import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from linear_attention_serving_fwd_gb300 import _native, kv_cache


class Fake(torch.Tensor):
    """A CPU tensor that says it is on CUDA device ``index``."""
    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


def fake(t, index=0):
    t = t.as_subclass(Fake)
    t.index = index
    return t


class Library:
    """Notes the calls' names; every call succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 1 << 16 if name == "kda_paged_attention_workspace_bytes" else 0
        return call


class Stream:
    cuda_stream = 0x77

    def __init__(self, index=0):
        self.device = torch.device("cuda", index)


@pytest.fixture
def world(monkeypatch):
    """The library, and the stream that each tensor of a call was made on (None:
    the current one)."""
    w = types.SimpleNamespace(lib=Library(), made=[], current=None, device=0)

    @contextlib.contextmanager
    def on(stream):
        before, w.current = w.current, stream
        yield
        w.current = before

    def making(make):
        def f(*args, device=None, **kw):
            w.made.append(w.current)
            return fake(make(*args, **kw))
        return f

    monkeypatch.setattr(_native, "lib", lambda: w.lib)
    monkeypatch.setattr(kv_cache, "_raw_stream", lambda device: w.current.cuda_stream if w.current else 0x55)
    monkeypatch.setattr(kv_cache, "_current_device", lambda: w.device)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(kv_cache.torch, "empty", making(torch.empty))
    monkeypatch.setattr(kv_cache.torch, "zeros", making(torch.zeros))
    return w


def _i32(*shape):
    return fake(torch.ones(shape, dtype=torch.int32))


def _pages():
    return kda.KvPages(_i32(2), _i32(2, 4), _i32(8), _i32(1), 16)


def _cache():
    kv = torch.ones(2, 8, 16, 2, 128, dtype=torch.bfloat16)
    return kda.KvCache(fake(kv[0]), fake(kv[1]))


def _rows(t, heads):
    return fake(torch.ones(t, heads, 128, dtype=torch.bfloat16))


@pytest.mark.parametrize("stream", [None, Stream()])
def test_what_a_call_makes_belongs_to_its_stream(world, stream):
    """Memory from the current stream's pool would be handed on, or still be in
    use, in that stream's order and not in the call's."""
    handle = 0x77 if stream else 0x55
    kda.kda_kv_extend(_pages(), _i32(2), 3, stream=stream)
    assert world.made == [stream] * 3 and world.lib.calls[-1][1][-1] == handle
    kda.kda_paged_attention(_cache(), _rows(3, 4), _i32(3), _i32(2), _i32(2, 4), return_lse=True, stream=stream)
    assert world.made == [stream] * 6 and world.lib.calls[-1][1][-1] == handle
    assert world.current is None
    # what the caller brings stays the caller's
    kda.kda_kv_extend(_pages(), _i32(2), 3, cu_seqlens=_i32(3), slot_map=_i32(3), step_lens=_i32(2), stream=stream)
    ws = fake(torch.ones(1 << 16, dtype=torch.uint8))
    kda.kda_paged_attention(_cache(), _rows(3, 4), _i32(3), _i32(2), _i32(2, 4), out=_rows(3, 4), workspace=ws,
                            stream=stream)
    assert len(world.made) == 6


def _calls():
    """Each call, its tensors by name."""
    pages, cache = _pages(), _cache()
    return [
        (lambda **t: kda.kda_kv_extend(pages, t.pop("new_lens"), 3, **t),
         dict(new_lens=_i32(2), cu_seqlens=_i32(3), slot_map=_i32(3), step_lens=_i32(2))),
        (lambda **t: kda.kda_kv_truncate(pages, t.pop("keep_lens"), **t), dict(keep_lens=_i32(2))),
        (lambda **t: kda.kda_kv_append(cache, t.pop("k"), t.pop("v"), t.pop("slot_map"), **t),
         dict(k=_rows(3, 2), v=_rows(3, 2), slot_map=_i32(3))),
        (lambda **t: kda.kda_paged_attention(cache, t.pop("q"), t.pop("cu_seqlens"), t.pop("kv_lens"), t.pop("block_table"), **t),
         dict(q=_rows(3, 4), cu_seqlens=_i32(3), kv_lens=_i32(2), block_table=_i32(2, 4), out=_rows(3, 4),
              lse=fake(torch.ones(3, 4)), workspace=fake(torch.ones(1 << 16, dtype=torch.uint8)))),
    ]


def test_tensors_of_another_device_are_refused(world):
    for call, tensors in _calls():
        call(**tensors)
        done = len(world.lib.calls)
        for name, t in tensors.items():
            with pytest.raises(ValueError, match=f"{name}.*cuda:0"):
                call(**{**tensors, name: fake(t.as_subclass(torch.Tensor), 1)})
        assert len(world.lib.calls) == done


def test_handles_of_two_devices_are_refused(world):
    good = [_i32(2), _i32(2, 4), _i32(8), _i32(1)]
    for i in range(1, 4):
        with pytest.raises(ValueError, match="cuda:0"):
            kda.KvPages(*good[:i], fake(good[i].as_subclass(torch.Tensor), 1), *good[i + 1:], 16)
    kv = torch.ones(2, 8, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="one device"):
        kda.KvCache(fake(kv[0]), fake(kv[1], 1))


def test_the_current_device_and_the_stream_are_the_handles(world):
    for call, tensors in _calls():
        done = len(world.lib.calls)
        with pytest.raises(ValueError, match="stream.*cuda:0"):
            call(**tensors, stream=Stream(1))
        world.device = 1
        with pytest.raises(ValueError, match="current device.*cuda:0"):
            call(**tensors)
        world.device = 0
        assert len(world.lib.calls) == done
        call(**tensors, stream=Stream(0))
