"""Rotary positions against the fp64 oracle.

Tolerance, element by element: the result is rounded once to the 16-bit type,
half a step, u |y| with u = eps / 2 (and half of fp16's smallest number); before
that, cosine and sine are within 2 units of 2^-24 of a number of at most 1, the
products and their sum round at 2^-24: 8 * 2^-24 r (1 + u) with r = |x| + |y| of
the pair, times the amplitude.  The oracle's own angle p f is rounded to 53 bits: p f 2^-53 r."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from oracle import quant

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rnd(*s, dtype=BF16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*s, generator=g, device="cuda").to(dtype)


def _check(got, x, positions, rope, freqs):
    a, xd = rope.amplitude, x.double().cpu().numpy()
    want = quant.rope(xd, positions, freqs, rope.layout, a)
    n = len(freqs)
    r = np.abs(xd).copy()
    i, j = (np.arange(n), np.arange(n) + n) if rope.layout == "half" else (np.arange(n) * 2, np.arange(n) * 2 + 1)
    r[..., i] = r[..., j] = np.abs(xd[..., i]) + np.abs(xd[..., j])
    u = torch.finfo(x.dtype).eps / 2
    far = max([abs(p) for p in positions] + [1]) * max(map(abs, freqs))
    tol = u * np.abs(want) + abs(a) * r * (8 * 2.0 ** -24 + far * 2.0 ** -53) * (1 + u) + (2.0 ** -25 if x.dtype == FP16 else 0)
    stay = np.arange(128) >= 2 * n
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= tol).all(), (off - tol).max()
    assert torch.equal(got[..., torch.from_numpy(stay)], x[..., torch.from_numpy(stay).cuda()])
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("dim", [2, 4, 14, 16, 30, 32, 64, 96, 112, 126, 128])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_parts_of_the_head(dim, layout, dtype):
    f = kda.rope_frequencies(dim, 1e4)
    rope = kda.Rope(f, layout=layout)
    q, k = _rnd(9, 5, 128, dtype=dtype), _rnd(9, 2, 128, dtype=dtype, seed=1)
    pos = [0, 1, 2, 17, 1000, 4095, 65536, 1000000, 3]
    yq, yk = kda.kda_rope(rope, q, k, positions=_i32(pos))
    _check(yq, q, pos, rope, f.tolist())
    _check(yk, k, pos, rope, f.tolist())


@pytest.mark.parametrize("heads", [(1, 0), (1, 1), (3, 1), (8, 8), (24, 8), (33, 2), (96, 8), (0, 4)])
@pytest.mark.parametrize("tokens", [1, 7, 200])
def test_heads(heads, tokens):
    f = kda.rope_frequencies(128, 5e5, factor=4.0, original_context=8192)
    rope = kda.Rope(f, layout="half", amplitude=1.25)
    pos = np.random.default_rng(tokens).integers(0, 100000, tokens).tolist()
    both = _rnd(tokens, sum(heads) + 3, 128, seed=tokens)  # bands of a projection
    q, k = both[:, 1:1 + heads[0]], both[:, 2 + heads[0]:2 + sum(heads)]
    yq, yk = kda.kda_rope(rope, q, k if heads[1] else None, positions=_i32(pos))
    _check(yq, q, pos, rope, f.tolist())
    if heads[1]:
        _check(yk, k, pos, rope, f.tolist())


@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [5, 0, 0, 300, 1, 0], [0, 2], [1] * 33, [2] * 1100, [0] * 40 + [3] + [0] * 70])
def test_positions_of_requests(lens):
    r = np.random.default_rng(len(lens))
    kv = [n + int(r.integers(0, 5000)) for n in lens]
    pos = [v - n + i for n, v in zip(lens, kv) for i in range(n)]
    f = kda.rope_frequencies(64, 1e4)
    rope = kda.Rope(f, layout="pairs")
    q, k = _rnd(sum(lens) + 4, 2, 128), _rnd(sum(lens) + 4, 1, 128, seed=2)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    out = [torch.full_like(q, 7.0), torch.full_like(k, 7.0)]
    kda.kda_rope(rope, q, k, cu_seqlens=_i32(cu), kv_lens=_i32(kv), q_out=out[0], k_out=out[1])
    for x, y in zip((q, k), out):
        _check(y[:len(pos)], x[:len(pos)], pos, rope, f.tolist())
        assert (y[len(pos):] == 7).all()  # tokens of no request


def test_tokens_before_the_first_request_and_before_position_0():
    f = kda.rope_frequencies(128)
    rope = kda.Rope(f)
    q = _rnd(8, 2, 128)
    out = torch.full_like(q, 7.0)
    kda.kda_rope(rope, q, cu_seqlens=_i32([2, 4, 7]), kv_lens=_i32([0, 2]), q_out=out)  # a request that was not admitted
    pos = [-2, -1, -1, 0, 1]
    _check(out[2:7], q[2:7], pos, rope, f.tolist())
    assert (out[:2] == 7).all() and (out[7:] == 7).all()


@pytest.mark.parametrize("dim", [128, 64, 30])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_in_place(dim, layout):
    rope = kda.Rope(kda.rope_frequencies(dim), layout=layout)
    both = _rnd(300, 12, 128)
    before = both.clone()
    q, k = both[:, :8], both[:, 8:10]
    pos = _i32(list(range(50, 350)))
    want = kda.kda_rope(rope, q, k, positions=pos)
    got = kda.kda_rope(rope, q, k, positions=pos, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(both[:, 10:], before[:, 10:])


def test_far_positions_and_fast_pairs():
    """An angle of 2^31 turns and a fraction: what a product in 32 bits has lost."""
    f = [3.0, 0.1, 1e-9, 2.0 ** -40]
    rope = kda.Rope(f)
    q = _rnd(3, 1, 128)
    pos = [2 ** 31 - 1, 2 ** 30 + 1, 99999999]
    _check(kda.kda_rope(rope, q, positions=_i32(pos))[0], q, pos, rope, f)


def test_head_major_outputs():
    rope = kda.Rope(kda.rope_frequencies(128))
    q = _rnd(40, 4, 128)
    out = torch.zeros(4, 40, 128, dtype=BF16, device="cuda").transpose(0, 1)
    kda.kda_rope(rope, q, positions=_i32(list(range(40))), q_out=out)
    assert torch.equal(out, kda.kda_rope(rope, q, positions=_i32(list(range(40))))[0])


def test_nothing_to_turn():
    rope = kda.Rope(kda.rope_frequencies(128))
    q = _rnd(0, 4, 128)
    assert kda.kda_rope(rope, q, positions=_i32([]))[0].shape == (0, 4, 128)
    x = _rnd(3, 4, 128)
    out = torch.full_like(x, 7.0)
    kda.kda_rope(rope, x, cu_seqlens=_i32([0]), kv_lens=_i32([]), q_out=out)
    assert (out == 7).all()


def test_graph_and_stream():
    rope = kda.Rope(kda.rope_frequencies(128))
    q, k, pos = _rnd(64, 8, 128), _rnd(64, 2, 128, seed=1), _i32(list(range(64)))
    out = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        kda.kda_rope(rope, q, k, positions=pos, q_out=out[0], k_out=out[1])
    q.copy_(_rnd(64, 8, 128, seed=5))
    pos += 100
    g.replay()
    torch.cuda.synchronize()
    want = kda.kda_rope(rope, q, k, positions=pos)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
