"""The Python side of the 8-bit cache's and the rotation's calls, without a GPU,
on the fakes of the 16-bit cache's test."""
from __future__ import annotations

import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda

from .test_kv_binding import Stream, _cache, _i32, _rows, fake, world  # noqa: F401

BF16 = torch.bfloat16


def _eight():
    x = torch.full((2, 8, 16, 2, 128), 0, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(2, 8, 2, 1)
    return kda.KvCache(fake(x[0]), fake(x[1]), fake(s[0]), fake(s[1]), dtype=BF16)


def _rope():
    r = kda.Rope.__new__(kda.Rope)
    r._index, r._ref, r.amplitude, r.layout = 0, None, 1.0, "half"
    return r


def test_calls_go_by_what_the_cache_holds(world):  # noqa: F811
    args = _rows(3, 2), _rows(3, 2), _i32(3)
    for cache, tail in ((_cache(), ""), (_eight(), "_quant")):
        kda.kda_kv_append(cache, *args)
        assert world.lib.calls[-1][0] == "kda_kv_append" + tail
        kda.kda_kv_read(cache, _i32(3))
        assert world.lib.calls[-1][0] == "kda_kv_read" + tail
        kda.kda_paged_attention(cache, _rows(3, 4), _i32(3), _i32(2), _i32(2, 4))
        assert world.lib.calls[-1][0] == "kda_paged_attention" + tail
        assert world.lib.calls[-2][0] == f"kda_paged_attention{tail}_workspace_bytes"


@pytest.mark.parametrize("stream", [None, Stream()])
def test_what_a_call_makes_belongs_to_its_stream(world, stream):  # noqa: F811
    handle = 0x77 if stream else 0x55
    kda.kda_kv_read(_eight(), _i32(3), stream=stream)
    assert world.made == [stream] * 2 and world.lib.calls[-1][1][-1] == handle
    kda.kda_rope(_rope(), _rows(3, 4), _rows(3, 2), positions=_i32(3), stream=stream)
    assert world.made == [stream] * 4 and world.lib.calls[-1][1][-1] == handle
    kda.kda_paged_attention(_eight(), _rows(3, 4), _i32(3), _i32(2), _i32(2, 4), return_lse=True, stream=stream)
    assert world.made == [stream] * 7 and world.current is None
    kda.kda_kv_read(_eight(), _i32(3), k=_rows(3, 2), v=_rows(3, 2), stream=stream)
    q = _rows(3, 4)
    kda.kda_rope(_rope(), q, positions=_i32(3), q_out=q, stream=stream)
    assert len(world.made) == 7


def _calls():
    cache = _eight()
    return [
        (lambda **t: kda.kda_kv_append(cache, t.pop("k"), t.pop("v"), t.pop("slot_map"), **t),
         dict(k=_rows(3, 2), v=_rows(3, 2), slot_map=_i32(3))),
        (lambda **t: kda.kda_kv_read(cache, t.pop("slot_map"), **t), dict(slot_map=_i32(3), k=_rows(3, 2), v=_rows(3, 2))),
        (lambda **t: kda.kda_paged_attention(cache, t.pop("q"), t.pop("cu_seqlens"), t.pop("kv_lens"), t.pop("block_table"), **t),
         dict(q=_rows(3, 4), cu_seqlens=_i32(3), kv_lens=_i32(2), block_table=_i32(2, 4), out=_rows(3, 4),
              lse=fake(torch.ones(3, 4)), workspace=fake(torch.ones(1 << 16, dtype=torch.uint8)))),
        (lambda **t: kda.kda_rope(_rope(), t.pop("q"), t.pop("k"), **t),
         dict(q=_rows(3, 4), k=_rows(3, 2), positions=_i32(3), q_out=_rows(3, 4), k_out=_rows(3, 2))),
        (lambda **t: kda.kda_rope(_rope(), t.pop("q"), **t), dict(q=_rows(3, 4), cu_seqlens=_i32(3), kv_lens=_i32(2))),
    ]


def test_tensors_of_another_device_are_refused(world):  # noqa: F811
    for call, tensors in _calls():
        call(**tensors)
        done = len(world.lib.calls)
        for name, t in tensors.items():
            with pytest.raises(ValueError, match=f"{name}.*cuda:0"):
                call(**{**tensors, name: fake(t.as_subclass(torch.Tensor), 1)})
        assert len(world.lib.calls) == done


def test_the_current_device_and_the_stream_are_the_handles(world):  # noqa: F811
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


def test_the_handles_rules(world):  # noqa: F811
    x = fake(torch.full((8, 16, 2, 128), 0, dtype=torch.uint8).view(torch.float8_e4m3fn))
    s = fake(torch.ones(8, 2, 1))
    with pytest.raises(TypeError, match="dtype"):
        kda.KvCache(x, x, s, s)
    with pytest.raises(TypeError, match="dtype"):
        kda.KvCache(x, x, s, s, dtype=torch.float32)
    for bad in (None, fake(torch.ones(8, 1, 2)), fake(torch.ones(8, 2, 1, dtype=torch.float64)), fake(torch.ones(8, 2, 1), 1)):
        with pytest.raises(ValueError, match="k_scale"):
            kda.KvCache(x, x, bad, s, dtype=BF16)
        with pytest.raises(ValueError, match="v_scale"):
            kda.KvCache(x, x, s, bad, dtype=BF16)
    wide = fake(torch.full((8, 16, 2, 128), 0, dtype=BF16))
    with pytest.raises(ValueError, match="16-bit"):
        kda.KvCache(wide, wide, s, s)
    with pytest.raises(ValueError, match="16-bit"):
        kda.KvCache(wide, wide, dtype=torch.float16)
    assert kda.KvCache(wide, wide, dtype=BF16).dtype == BF16 and not kda.KvCache(wide, wide).quantized


def test_the_rotations_rules(world):  # noqa: F811
    r, q, k = _rope(), _rows(3, 4), _rows(3, 2)
    with pytest.raises(ValueError, match="needed"):
        kda.kda_rope(r, q, k)
    with pytest.raises(ValueError, match="needed"):
        kda.kda_rope(r, q, k, cu_seqlens=_i32(3))
    with pytest.raises(ValueError, match="not both"):
        kda.kda_rope(r, q, k, positions=_i32(3), cu_seqlens=_i32(3), kv_lens=_i32(2))
    with pytest.raises(ValueError, match="same number"):
        kda.kda_rope(r, q, _rows(4, 2), positions=_i32(3))
    with pytest.raises(ValueError, match="shape"):
        kda.kda_rope(r, q, k, positions=_i32(3), q_out=_rows(3, 2))
    with pytest.raises(ValueError, match="without"):
        kda.kda_rope(r, q, positions=_i32(3), k_out=k)
    with pytest.raises(TypeError):
        kda.kda_rope(r, fake(torch.ones(3, 4, 128)), positions=_i32(3))
    with pytest.raises(TypeError):
        kda.kda_rope(r, q, fake(torch.ones(3, 2, 128, dtype=torch.float16)), positions=_i32(3))
    with pytest.raises(ValueError, match="entries"):
        kda.kda_rope(r, q, k, positions=_i32(4))
