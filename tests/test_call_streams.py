"""The recurrent calls' tensors of their own on a stream that is passed in,
without a GPU: the fakes of the paged cache's binding tests."""
from __future__ import annotations

import types

import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from tests.test_kv_binding import Stream, _i32, _rows, fake, world  # noqa: F401

T, H, W = 3, 2, 4


def _args():
    beta = fake(torch.ones(T, H, dtype=torch.bfloat16))
    return [_rows(T, H) for _ in range(4)] + [beta]


def _pool():
    return fake(torch.ones(2, H, 128, 128))


def _records():
    return fake(torch.ones(1, H, W, 128)), fake(torch.ones(1, H, W, 256, dtype=torch.bfloat16))


CALLS = {  # and what each makes: output, states, workspace, records, counter
    "kda_chunk_fwd": (lambda **kw: kda.kda_chunk_fwd(*_args(), output_final_state=True, **kw), 3),
    "kda_chunk_fwd_noalloc": (lambda **kw: kda.kda_chunk_fwd_noalloc(*_args(), out=_rows(T, H), **kw), 0),
    "kda_decode": (lambda **kw: kda.kda_decode(*_args(), _pool(), _i32(2), _i32(1), W, **kw), 1),
    "kda_decode_steps": (lambda **kw: kda.kda_decode_steps(*_args(), _pool(), _i32(2), _i32(1, W), W, **kw), 1),
    "kda_verify": (lambda **kw: kda.kda_verify(*_args(), _pool(), _i32(2), _i32(1), W, **kw), 4),
    "kda_commit": (lambda **kw: kda.kda_commit(_pool(), _i32(1), _i32(1), *_records(), W, **kw), 0),
}


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_belongs_to_its_stream(world, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: world.current or types.SimpleNamespace(cuda_stream=0x55))
    call, made = CALLS[name]
    for stream, handle in ((None, 0x55), (Stream(), 0x77)):
        world.made.clear()
        call(stream=stream)
        assert world.made == [stream] * made and world.current is None
        assert world.lib.calls[-1][1][-1].value == handle


@pytest.mark.gpu
def test_calls_on_another_stream_wait_for_nothing_of_the_current_one():
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    n, h = 320, 4
    x = [rnd(n, h, 128) for _ in range(4)] + [rnd(n, h)]
    gate = dict(A_log=torch.zeros(h, device="cuda"), dt_bias=torch.zeros(h, 128, device="cuda"))
    pool = torch.randn(80, h, 128, 128, generator=g, device="cuda")
    starts = torch.arange(0, n + 1, 4, dtype=torch.int32, device="cuda")
    slots = torch.arange(80, dtype=torch.int32, device="cuda")

    def calls(**kw):
        return [*kda.kda_chunk_fwd(*x, output_final_state=True, **gate, **kw),
                *kda.kda_verify(*x, pool, starts, slots, 4, **gate, **kw)]

    s = torch.cuda.Stream()
    want = calls()
    calls(stream=s)  # kernels are loaded and pools grown
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    got = calls(stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and kda.kda_device_status() == 0
