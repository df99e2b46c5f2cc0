"""The 8-bit cache's append and read-back against the fp64 oracle.  Scales are
powers of two and every number is rounded once to nearest-even (a grown block's
earlier rows once more), so everything is equal bit for bit."""
from __future__ import annotations

import random

import numpy as np
import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from oracle import quant

pytestmark = pytest.mark.gpu
INDEX = 5
BF16, FP16, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _np(x):
    return x.double().cpu().numpy()


class Pool:
    """A cache with random contents, and the same as fp64 arrays."""

    def __init__(self, n_pages, page, heads, dtype=BF16, layout="tokens", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (n_pages, heads, page, 128) if layout == "heads" else (n_pages, page, heads, 128)
        if layout == "pairs":
            both = torch.randint(0, 256, (n_pages, 2, page, heads, 128), generator=g, device="cuda", dtype=torch.uint8)
            k, v = both[:, 0], both[:, 1]
        else:
            k, v = (torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
            if layout == "heads":
                k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
        for x in (k, v):
            x[(x & 0x7f) == 0x7f] = 3  # no NaN
        e = torch.randint(-12, 3, (2, n_pages, heads, page // 16), generator=g, device="cuda")
        self.scales = torch.exp2(e.float())
        self.cache = kda.KvCache(k.view(F8), v.view(F8), self.scales[0], self.scales[1], dtype=dtype)
        self.page, self.heads, self.dtype = page, heads, dtype
        self.want = [_np(self.cache.k), _np(self.scales[0]), _np(self.cache.v), _np(self.scales[1])]

    def rows(self, t, gain=1.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(t, 2 * self.heads + 1, 128, generator=g, device="cuda") * gain
        x = (x * torch.exp(torch.randn(t, 2 * self.heads + 1, 1, generator=g, device="cuda"))).to(self.dtype)
        return x[:, :self.heads], x[:, self.heads:2 * self.heads]  # bands of a projection

    def append(self, k, v, slots):
        kda.kda_kv_append(self.cache, k, v, _i32(slots))
        quant.append(self.want[0], self.want[1], _np(k), slots)
        quant.append(self.want[2], self.want[3], _np(v), slots)

    def same(self):
        c = self.cache
        for got, want in zip((c.k, c.k_scale, c.v, c.v_scale), self.want):
            got = _np(got)
            assert np.array_equal(got, want, equal_nan=True), np.argwhere((got != want) & ~np.isnan(want))[:4]
        assert kda.kda_device_status() == 0


@pytest.mark.parametrize("page,layout,dtype", [(16, "tokens", BF16), (32, "heads", FP16), (64, "pairs", BF16), (256, "tokens", FP16),
                                               (128, "heads", BF16)])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_steps_of_a_batch(page, layout, dtype, heads):
    """Requests grow by ragged numbers of tokens, in pages of a random order."""
    r = random.Random(page + heads)
    n_req, n_pages = 9, 9 * (-(-600 // page))
    p = Pool(n_pages, page, heads, dtype, layout, seed=page)
    ids = list(range(n_pages))
    r.shuffle(ids)
    table = [[ids.pop() for _ in range(-(-600 // page))] for _ in range(n_req)]
    lens = [0] * n_req
    for step in range(6):
        new = [r.choice([0, 1, 1, 4, 15, 16, 17, 90]) for _ in range(n_req)]
        slots = [-1 if r.random() < 0.02 and n == 1 else table[b][q // page] * page + q % page
                 for b, n in enumerate(new) for q in range(lens[b], lens[b] + n)]
        k, v = p.rows(len(slots), gain=10.0 ** r.randint(-3, 2), seed=step)
        p.append(k, v, slots)
        lens = [a + n for a, n in zip(lens, new)]
        lens = [r.choice([x, max(0, x - 3)]) for x in lens]  # rejected drafts: rows written anew
    p.same()


@pytest.mark.parametrize("tokens", [1, 2, 500, 5000])
def test_whole_prompts(tokens):
    p = Pool(-(-tokens // 64) + 1, 64, 2, seed=tokens)
    p.append(*p.rows(tokens, seed=tokens), list(range(64, 64 + tokens)))
    p.same()


@pytest.mark.parametrize("window", range(1, 17))
def test_windows_that_cross_blocks(window):
    p = Pool(40, 16, 2, FP16, seed=window)
    slots = [b * 32 + 7 + i for b in range(19) for i in range(window)]
    p.append(*p.rows(len(slots), seed=window), slots)
    p.same()


def test_values_at_the_borders():
    for dtype, big in ((BF16, [3e38, 1e20, 2.0 ** 56, 1.27e17]), (FP16, [65504.0, 448.0, 449.0])):
        for m in big + [1e-30, 2.0 ** -24, 1.75, 1.7578125, 0.0, 448.0, 224.0, 2.0 ** -48, 1e-20]:
            p = Pool(1, 16, 1, dtype)
            k, v = p.rows(3)
            k = k.clone().zero_()
            k[1, 0, 5], k[2, 0, 127], k[0, 0, 0] = m, -m / 3, m / 200
            p.append(k, v, [5, 6, 7])
            p.same()
            p.append(v, k, [0, 1, 2])  # a block that begins anew
            p.same()


def test_infinities_and_nan():
    """Only finite numbers set a scale; infinities become the largest number, NaN stays."""
    for dtype in (BF16, FP16):
        p = Pool(2, 16, 2, dtype)
        k, v = (x.clone() for x in p.rows(6))
        k[0, 0, 3], k[1, 0, 4], k[2, 1, 5], v[3, 0, 6] = float("inf"), float("-inf"), float("nan"), float("nan")
        v[:, 1] = float("inf")  # nothing finite at all
        p.append(k, v, [16, 17, 18, 19, 20, 21])
        assert p.want[0][1, 0, 0, 3] == 448 and np.isnan(p.want[0][1, 2, 1, 5]) and p.want[3][1, 1, 0] == 2.0 ** -48
        p.same()


def test_scales_that_are_no_powers_of_two():
    """A cache filled elsewhere: numbers go in by the scale's reciprocal in fp32, within a rounding of it."""
    p = Pool(2, 16, 1, seed=4)
    p.scales[:] = 0.3
    k, v = p.rows(2, gain=0.5)
    kda.kda_kv_append(p.cache, k, v, _i32([5, 6]))
    inv = np.float32(1) / np.float32(0.3)
    assert torch.equal(p.scales[:, 0].cpu(), torch.full((2, 1, 1), 0.3))
    assert np.array_equal(_np(p.cache.k)[0, 5:7], quant.round_e4m3(_np((k.float() * float(inv)))))
    big = k.float().mul(1e4).to(BF16)
    before = _np(p.cache.k)[0, :7] * float(np.float32(0.3))
    kda.kda_kv_append(p.cache, big, v, _i32([7, 8]))
    scale = 2.0 ** quant.exponent(float(big.abs().max()))
    assert float(p.scales[0, 0, 0, 0]) == scale
    after = _np(p.cache.k)[0, :7] * scale
    # half a step, and what the number times the ratio of the scales, two roundings to 24 bits, may be
    # past it: 0.3 is no fp32 number, and 1.875 * 0.3 = 4.5 of 64 * 2^-9 lands on the tie from above
    half = np.maximum(2.0 ** -4 * np.abs(before), scale * 2.0 ** -10)
    assert (np.abs(after - before) <= half + 2.0 ** -22 * np.abs(before)).all()


def test_bad_slots_are_reported():
    p = Pool(4, 16, 2)
    k, v = p.rows(6)
    kda.kda_kv_append(p.cache, k, v, _i32([64, 17, 18, 18, 19, 1 << 30]))  # past the cache; a slot twice
    assert kda.kda_device_status() == INDEX
    for i, x in ((0, k), (2, v)):
        quant.append(p.want[i], p.want[i + 1], _np(x)[1:3], [17, 18])
    p.same()


def test_extend_gives_the_slots():
    pages = kda.KvPages.empty(3, 8, 24, 32)
    p = Pool(24, 32, 2)
    for new in ([5, 40, 1], [1, 1, 1], [4, 4, 60]):
        _, slots, _ = kda.kda_kv_extend(pages, _i32(new), sum(new))
        p.append(*p.rows(sum(new), seed=new[2]), slots.tolist())
    p.same()


@pytest.mark.parametrize("page,layout,dtype", [(16, "tokens", BF16), (64, "heads", FP16), (256, "pairs", BF16)])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (7, 3), (1000, 8)])
def test_read(page, layout, dtype, tokens, heads):
    n_pages = -(-tokens // page) + 2
    p = Pool(n_pages, page, heads, dtype, layout, seed=tokens)
    g = random.Random(tokens)
    slots = [g.choice([-1, g.randrange(n_pages * page)]) for _ in range(tokens)]
    k, v = kda.kda_kv_read(p.cache, _i32(slots))
    for got, x, s in ((k, p.want[0], p.want[1]), (v, p.want[2], p.want[3])):
        want = torch.from_numpy(quant.values(x, s)).to(dtype).reshape(-1, heads, 128)
        want = torch.stack([want[i] if i >= 0 else torch.zeros_like(want[0]) for i in slots])
        assert torch.equal(got.cpu(), want)
    assert kda.kda_device_status() == 0


def test_read_of_a_16_bit_cache():
    for dtype in (BF16, FP16):
        kv = torch.randn(2, 5, 2, 64, 128, device="cuda").to(dtype).permute(0, 1, 3, 2, 4)  # head-major
        cache = kda.KvCache(kv[0], kv[1])
        slots = _i32([0, 5, -1, 319, 64, 5])
        k, v = kda.kda_kv_read(cache, slots)
        for got, x in ((k, kv[0]), (v, kv[1])):
            want = x.reshape(-1, 2, 128)[slots.long().clamp(min=0)]
            want[2] = 0
            assert torch.equal(got, want)


def test_read_past_the_cache():
    p = Pool(2, 16, 2)
    k, v = kda.kda_kv_read(p.cache, _i32([3, 32]))
    assert kda.kda_device_status() == INDEX and not k[1].any() and not v[1].any() and k[0].any()


def test_read_inverts_append():
    cache = kda.KvCache.empty(8, 64, 2, quantized=True)
    k, v = (torch.randn(300, 2, 128, device="cuda").bfloat16() for _ in range(2))
    slots = _i32(list(range(300)))
    kda.kda_kv_append(cache, k, v, slots)
    got = kda.kda_kv_read(cache, slots)
    for x, y in zip((k, v), got):
        m = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, 4)).view(19, 16, 2, 128).abs().amax((1, 3))  # of each block
        m = m.repeat_interleave(16, 0)[:300, :, None]
        # half a step of 4 bits; below the normal range half of 2^-9 of a scale of at most m / 224
        assert ((x.float() - y.float()).abs() <= torch.maximum(x.float().abs() * 2.0 ** -4, m / 224 * 2.0 ** -10)).all()
    kda.kda_kv_append(cache, got[0], got[1], slots)  # what has been rounded stays
    again = kda.kda_kv_read(cache, slots)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_captured_and_replayed():
    p = Pool(8, 16, 2)
    k, v = (x.contiguous() for x in p.rows(8))
    slots = _i32(list(range(32, 40)))
    out = torch.empty_like(k), torch.empty_like(v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_kv_append(p.cache, k, v, slots)
        kda.kda_kv_read(p.cache, slots, k=out[0], v=out[1])
    k.copy_(p.rows(8, seed=9)[0])
    g.replay()
    torch.cuda.synchronize()
    for i, x in ((0, k), (2, v)):
        quant.append(p.want[i], p.want[i + 1], _np(x), slots.tolist())
    p.same()
    want = quant.values(p.want[0], p.want[1]).reshape(-1, 2, 128)[32:40]
    assert np.array_equal(_np(out[0]), want)


def test_empty_calls():
    p = Pool(1, 16, 1)
    p.append(*p.rows(0), [])
    k, v = kda.kda_kv_read(p.cache, _i32([]))
    assert k.shape == (0, 1, 128)
    p.same()
