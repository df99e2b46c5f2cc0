"""Attention over the 8-bit cache against the fp64 oracle on the numbers that the
cache stands for.

Tolerance, element by element, with u = eps / 2 of the 16-bit type.  The output
is rounded to that type once: u |o|.  A weight is rounded to fp16 (2^-11) and
taken in parts of 3 significant bits each: two parts (bf16) leave at most 2^-7 of
it, three (fp16) 2^-10: w W, W = sum_j p_j |v_j| with the normalised p, and w =
2^-7 + 2^-11 or 2^-10 + 2^-11.  Below the normal range a weight is off by at most 2^-17
where the largest is at least 2^7 (as weight times scale): 2^-24 of the largest
per key, n 2^-23 max|v|.  The 32-bit steps: a query row in 8-bit parts is off by
at most 2^-17 of its largest element per element, and a score's 3 * 128 additions by 2^-24 of
sum |q_i k_i| each: with R = max over the case of scale |q|_max |k|_1 (which bounds sum |q_i k_i| scale),
e = (2^-17 + 384 * 2^-24) R, so p is off by e and the sum as well: 2 e W, and e + 2^-13 + 2^-22 |lse|
for the lse (2^-13: the exponential and logarithm of sums of up to 2^15 weights).  Rows
that see nothing are exactly 0 and -inf."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from oracle import paged, quant

pytestmark = pytest.mark.gpu
INDEX, RANGE = 5, 6
BF16, FP16, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _np(x):
    return x.double().cpu().numpy()


def _bytes(shape, g):
    """Random numbers of the 8-bit type, most of them in its upper octaves, as bytes."""
    return (torch.randn(shape, generator=g, device="cuda") * 90).clamp(-448, 448).to(F8).view(torch.uint8)


class Case:
    """new, kv: tokens of each request and its cached tokens, these included."""

    def __init__(self, new, kv, hq, hkv, page, dtype=BF16, layout="tokens", seed=0, gain=1.0, extra_cols=1, cols=None,
                 spread=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        owned = [-(-n // page) for n in kv]
        n_pages = sum(owned) + 2
        if layout == "pairs":
            both = _bytes((n_pages, 2, page, hkv, 128), g)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            shape = (n_pages, hkv, page, 128) if layout == "heads" else (n_pages, page, hkv, 128)
            self.k, self.v = _bytes(shape, g), _bytes(shape, g)
            if layout == "heads":
                self.k, self.v = self.k.permute(0, 2, 1, 3), self.v.permute(0, 2, 1, 3)
        self.k, self.v = self.k.view(F8), self.v.view(F8)
        e = torch.randint(-7 - spread, -6 + spread, (2, n_pages, hkv, page // 16), generator=g, device="cuda")
        self.ks, self.vs = torch.exp2(e[0].float().clamp(max=-6)), torch.exp2(e[1].float())
        ids = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        cols = cols or max(owned + [1]) + extra_cols
        self.table = [[ids.pop() for _ in range(n)] + [-1] * (cols - n) for n in owned]
        t = sum(new)
        self.q = (torch.randn(t, hq + 2, 128, generator=g, device="cuda") * gain).to(dtype)[:, 1:hq + 1]
        self.cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.new, self.kv, self.page, self.dtype, self.scale = new, list(kv), page, dtype, 128 ** -0.5

    def rows(self, b):
        return [(self.table[b][j // self.page], j % self.page) for j in range(self.kv[b])]

    def cache(self):
        return kda.KvCache(self.k, self.v, self.ks, self.vs, dtype=self.dtype)

    def set(self, x, at, value):
        """A number of the cache: x is self.k or self.v, ``at`` an index of [page, row, head, dim]."""
        x.view(torch.uint8)[at] = torch.tensor(float(value)).to(F8).view(torch.uint8).item()

    def run(self, window=0, sinks=0, **kw):
        return kda.kda_paged_attention(self.cache(), self.q, _i32(self.cu), _i32(self.kv), _i32(self.table), scale=self.scale,
                                       window=window, sinks=sinks, return_lse=True, **kw)

    def numbers(self):
        return quant.values(_np(self.k), _np(self.ks)), quant.values(_np(self.v), _np(self.vs))

    def check(self, window=0, sinks=0, result=None, rows=slice(None), q=None, k=None, v=None, kv=None):
        out, lse = self.run(window, sinks) if result is None else result
        kn, vn = self.numbers()
        k, v = kn if k is None else k, vn if v is None else v
        q = _np(self.q) if q is None else q
        want, want_lse, weight = paged.attention(q, k, v, self.cu, self.kv if kv is None else kv, self.table, self.scale,
                                                 window, sinks)
        out, lse = _np(out)[rows], _np(lse)[rows]
        want, want_lse, weight = want[rows], want_lse[rows], weight[rows]
        u = torch.finfo(self.dtype).eps / 2
        w = (2.0 ** -7 if self.dtype == BF16 else 2.0 ** -10) + 2.0 ** -11
        fin = np.nan_to_num(k, nan=0.0)
        reach = self.scale * np.abs(np.nan_to_num(q)).max(initial=0) * np.abs(fin).sum(-1).max(initial=0)
        e = (2.0 ** -17 + 384 * 2.0 ** -24) * reach
        vmax = np.abs(np.nan_to_num(v, nan=0.0)).max(initial=0)
        tol = u * np.abs(want) + (w + 2 * e) * weight * (1 + u) + max(self.kv + [0]) * 2.0 ** -23 * vmax + 1e-30
        if self.dtype == FP16:
            tol += 2.0 ** -25
        empty = np.isneginf(want_lse)
        assert np.array_equal(empty, np.isneginf(lse)) and not out[empty].any()
        if self.dtype == FP16:
            # 8-bit numbers times scales reach past fp16: where want +- tol reaches a number that rounds past the
            # largest, 65504, an infinity of that sign is within it
            past = (np.isposinf(out) & (want + tol >= 65520)) | (np.isneginf(out) & (want - tol <= -65520))
            out, want = np.where(past, 0, out), np.where(past, 0, want)
            assert (np.abs(want) - tol < 65520).all()
        off = np.abs(out - want) - tol
        assert np.isfinite(out).all() and off.max(initial=-1) <= 0, f"{np.argmax(off)}: {off.max()}"
        lse_off = np.abs(lse[~empty] - want_lse[~empty]) - e - 2.0 ** -13 - 2.0 ** -22 * np.abs(want_lse[~empty])
        assert lse_off.max(initial=-1) <= 0, lse_off.max()
        assert kda.kda_device_status() == 0


# --- lengths, heads, pages, windows ---------------------------------------------

@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 385, 1000])
@pytest.mark.parametrize("dtype,layout,page", [(BF16, "tokens", 16), (FP16, "heads", 64), (BF16, "pairs", 256)])
def test_single_tokens(kv, dtype, layout, page):
    Case([1, 1], [kv, max(1, kv - 1)], 4, 2, page, dtype, layout, seed=kv).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (10, 2), (6, 1), (7, 1), (8, 1), (24, 2), (16, 1), (33, 1),
                                   (128, 1), (100, 1)])
@pytest.mark.parametrize("new,kv,dtype", [([1, 3], [200, 130], BF16), ([150], [150], FP16), ([40], [300], BF16)])
def test_head_groups(hq, hkv, new, kv, dtype):
    Case(new, kv, hq, hkv, 32, dtype, seed=hq).check()


@pytest.mark.parametrize("new,kv", [
    ([128], [128]), ([129], [129]), ([127], [127]), ([256], [256]), ([257], [257]), ([300], [300]), ([513], [513]),
    ([64], [1000]), ([200], [713]), ([5], [517]), ([1, 130, 2, 256, 1], [700, 130, 9, 600, 1]),
    ([0, 3, 0, 140, 0], [5, 3, 0, 270, 900]),
])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_chunks(new, kv, dtype):
    Case(new, kv, 2, 1, 64, dtype, seed=sum(kv)).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (100, 5), (128, 128), (300, 130), (1, 0), (1, 1), (40, 1000)])
def test_pages_and_windows(page, window, sinks):
    Case([70, 1, 4], [480, 611, 260], 3, 1, page, FP16 if page == 32 else BF16, "heads" if page > 64 else "tokens",
         seed=page).check(window, sinks)


@pytest.mark.parametrize("window,sinks", [(128, 4), (64, 0), (513, 16), (1, 0), (5000, 4)])
def test_windows_over_a_long_prompt(window, sinks):
    Case([1100], [1100], 2, 2, 64, seed=3).check(window, sinks)


@pytest.mark.parametrize("kv", [9000, 20000])
def test_one_long_cache(kv):
    Case([1], [kv], 4, 1, 64, seed=kv).check()
    Case([2], [kv], 4, 2, 128, FP16, seed=kv).check(window=4096, sinks=4)
    Case([3], [kv], 8, 1, 16, seed=kv).check()


def test_many_requests():
    r = np.random.default_rng(5)
    kv = r.integers(1, 500, 300)
    new = [int(min(n, r.choice([1, 1, 1, 2, 4]))) for n in kv]
    Case(new, kv.tolist(), 4, 2, 32, seed=5).check()
    Case(new, kv.tolist(), 4, 2, 32, FP16, seed=5).check(window=64, sinks=4)


def test_more_requests_than_a_block_counts():
    n = 3000
    Case([1] * n, [1 + i % 37 for i in range(n)], 1, 1, 16, seed=6).check()


# --- numbers ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("gain", [1e-4, 8.0, 40.0])
def test_sharp_and_flat_scores(gain, dtype):
    c = Case([3, 140], [900, 400], 2, 1, 64, dtype, seed=9, gain=gain)
    c.check()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("spread", [0, 12, 30])
def test_scales_that_differ(dtype, spread):
    """Values whose blocks' sizes lie octaves apart: the smaller ones' weights
    are tiny beside the others', but count in the sum."""
    c = Case([2, 150], [900, 700], 4, 2, 32, dtype, seed=spread, spread=spread)
    c.check()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_values_of_zero_and_of_the_smallest_scale(dtype):
    """Blocks whose values are all 0, with the least scale there is: their keys'
    weights are a large part of the sum."""
    c = Case([1, 140], [1000, 300], 2, 1, 16, dtype, seed=12)
    for pg in (c.table[0][:20] + c.table[1][3:6]):
        c.v.view(torch.uint8)[pg] = 0
        c.vs[pg] = 2.0 ** -48
    c.check()
    c.vs[c.table[0][30]] = 2.0 ** 48
    c.vs[c.table[1][1]] = 2.0 ** 40
    c.check()


@pytest.mark.parametrize("dtype,tol", [(BF16, 2.0 ** -7), (FP16, 2.0 ** -10)])
@pytest.mark.parametrize("gap", [0.0, 5.0, 9.0, 11.0, 12.5])
def test_a_needle_among_equals(gap, dtype, tol):
    """One key far above thousands of equal ones: each of their weights is tiny
    and all are off by the same rounding, but together they count.  Their values
    are 1, the needle's -1."""
    n = 20000
    c = Case([1], [n], 1, 1, 64, dtype, seed=13)
    c.q[...] = 1.0
    c.k.view(torch.uint8).zero_()
    c.ks[:], c.vs[:] = 1.0, 2.0 ** -7
    c.v.view(torch.uint8)[...] = torch.tensor(128.0).to(F8).view(torch.uint8).item()
    page, row = c.rows(0)[7777]
    c.set(c.k, (page, row, 0), 1.0)
    c.set(c.v, (page, row, 0), -128.0)
    c.scale = max(gap, 1e-6) / 128
    out, lse = c.run()
    others = (n - 1) * np.exp(-gap)
    want = (others - 1) / (others + 1)
    # the others' share is off by tol + 2^-11 at most, and what is left of it; the output's own rounding
    off = 2 * others / (1 + others) ** 2 * (tol + 2.0 ** -11) + others / (1 + others) * (tol + 2.0 ** -11)
    assert (np.abs(_np(out) - want) <= off + torch.finfo(dtype).eps / 2 * abs(want) + 1e-6).all()
    assert abs(float(lse) - np.log(np.exp(gap) + n - 1)) < 1e-4


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_scores_that_climb(dtype):
    """The reference moves many times, in some rows of a warp and not in others."""
    c = Case([2, 150], [1500, 700], 2, 1, 64, dtype, seed=31)
    c.q[::3] = torch.ones(128, device="cuda", dtype=dtype)
    c.ks[:] = 2.0 ** -5
    for b in range(2):
        rows = torch.tensor(c.rows(b), device="cuda")
        level = torch.arange(c.kv[b], device="cuda")[:, None] * 448 / 1500 + torch.randn(c.kv[b], 128, device="cuda")
        c.k.view(torch.uint8)[rows[:, 0], rows[:, 1], 0] = level.clamp(-448, 448).to(F8).view(torch.uint8)
    c.check()


def test_scales_that_are_no_powers_of_two():
    c = Case([2, 150], [700, 300], 4, 2, 32, BF16, seed=14)
    c.ks.mul_(torch.rand_like(c.ks) + 0.5)
    c.vs.mul_(torch.rand_like(c.vs) + 0.5)
    c.check()


def test_scales_out_of_range_are_reported():
    c = Case([1, 1], [300, 40], 1, 1, 64, seed=15)
    c.vs[c.table[0][1]] = 2.0 ** 60
    c.ks[c.table[0][2]] = float("nan")
    out = c.run()
    assert kda.kda_device_status(clear=True) == RANGE
    c.vs[c.table[0][1]], c.ks[c.table[0][2]] = 2.0 ** 48, 1.0
    c.check(result=out)


def test_queries_of_all_sizes():
    for dtype in (BF16, FP16):
        c = Case([1] * 8 + [40], [100] * 8 + [90], 2, 1, 16, dtype, seed=16)
        for i in range(6):
            c.q[i] *= 10.0 ** (i - 4)
        c.q[6] = 0.0
        c.q[7, 0, 3:] = 0.0
        c.check()


# --- rows that see nothing, hidden places ------------------------------------------

def test_rows_before_the_cache_begins():
    Case([5, 200, 3], [2, 130, 0], 2, 1, 16, seed=11).check()
    Case([300], [1], 4, 2, 64, FP16, seed=12).check(window=7, sinks=2)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("heads", [(1, 1), (4, 2), (3, 3), (6, 1)])
def test_blocks_without_keys(heads, dtype):
    """Whole blocks before position 0, of one tile and of two, wherever the cuts of
    the line of work fall in them, among blocks that have keys."""
    for extra in range(4):
        Case([300 + 37 * extra, 2, 70 + extra, 129], [1, 0, extra, 400], *heads, 16, dtype, seed=extra).check()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_hidden_places_have_no_influence(page, window, sinks, dtype):
    """NaN in hidden rows, and scales of blocks that no token sees."""
    c = Case([3, 140, 1], [50, 300, 413], 2, 1, page, dtype, seed=13)
    k, v = c.numbers()
    used = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    for b in range(3):
        for j, (pg, row) in enumerate(c.rows(b)):
            lo = c.kv[b] - c.new[b] + 1 - window if window else 0
            used[pg, row] = j >= lo or j < sinks
    c.k.view(torch.uint8)[~used] = 0x7f
    c.v.view(torch.uint8)[~used] = 0xff
    blocks = used.view(-1, page // 16, 16).any(-1)[:, None]
    for i, bad in enumerate((float("nan"), float("inf"), -1.0, 0.0)):
        (c.ks if i % 2 else c.vs)[~blocks] = bad
        c.check(window, sinks, k=k, v=v)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_poisoned_token_reaches_the_rows_that_see_it_alone(dtype):
    c = Case([200, 1], [260, 40], 2, 1, 32, dtype, seed=14)
    pg, row = c.rows(0)[60 + 77]  # position of token 77
    k, v = c.numbers()
    nan = float("nan")
    was = c.k.view(torch.uint8)[pg, row, 0, 9].item()
    c.set(c.v, (pg, row, 0, 5), nan)
    out, lse = c.run()
    c.check(result=(out, lse), rows=slice(0, 77), k=k, v=v)
    c.check(result=(out, lse), rows=slice(200, 201), k=k, v=v)
    assert torch.isnan(out[77:200, :, 5]).all() and torch.isfinite(lse[77:]).all()
    assert torch.isfinite(out[77:200, :, :5]).all() and torch.isfinite(out[77:200, :, 6:]).all()
    c.set(c.k, (pg, row, 0, 9), nan)
    out, lse = c.run()
    c.check(result=(out, lse), rows=slice(0, 77), k=k, v=v)
    assert torch.isnan(out[77:200]).all() and torch.isnan(lse[77:200]).all()
    c.k.view(torch.uint8)[pg, row, 0, 9] = was
    out, lse = c.run(window=30)
    seen = list(range(77)) + list(range(107, 201))
    c.check(window=30, result=(out, lse), rows=seen, k=k, v=v)


@pytest.mark.parametrize("new,kv", [([1, 1], [9000, 700]), ([2, 1], [300, 40]), ([150, 3], [700, 90]), ([300], [2600]),
                                    ([60] * 30, [500] * 30)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (250, 20), (1, 4)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_visible_values_that_are_nan(new, kv, window, sinks, dtype):
    c = Case(new, kv, 4, 2, 64, dtype, seed=71)
    last = kv[0] - new[0]
    for b, head, at, dim in [(0, 1, 3, 5), (0, 1, last, 9), (0, 1, max(0, last - 200), 10), (0, 1, kv[0] - 1, 11),
                             (0, 1, last + new[0] // 2, 12), (len(kv) - 1, 0, kv[-1] - 1, slice(None))]:
        page, row = c.rows(b)[at]
        c.set(c.v, (page, row, head, dim), float("nan"))
    out, lse = c.run(window, sinks)
    k, v = c.numbers()
    want, _, _ = paged.attention(_np(c.q), k, v, c.cu, c.kv, c.table, c.scale, window, sinks)
    clean = np.nan_to_num(v, nan=0.0)
    finite, _, _ = paged.attention(_np(c.q), k, clean, c.cu, c.kv, c.table, c.scale, window, sinks)
    bad = np.isnan(want)
    assert bad.any() and np.isnan(_np(out)[bad]).all()
    out = torch.where(torch.from_numpy(bad).cuda(), torch.from_numpy(finite).cuda(), out.double())
    c.check(window, sinks, result=(out, lse), v=clean)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("new,kv", [([1], [9000]), ([1], [200]), ([3], [5]), ([160], [5000]), ([20] * 40, [600] * 40)])
def test_a_query_that_is_not_finite(new, kv, value, dtype):
    c = Case(new, kv, 4, 2, 64, dtype, seed=51)
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[-1, 2] = bad[len(bad) // 2, 3] = True
    at = bad.nonzero(as_tuple=True)
    clean = _np(c.q)
    c.q[at[0], at[1], 17] = value
    out, lse = c.run()
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.isfinite(out[~bad]).all() and torch.isfinite(lse[~bad]).all()
    want, want_lse, _ = paged.attention(clean, *c.numbers(), c.cu, c.kv, c.table, c.scale)
    out, lse = torch.where(bad[..., None], torch.from_numpy(want).to(out), out), torch.where(bad, torch.from_numpy(want_lse).to(lse), lse)
    c.check(result=(out, lse), q=clean)


def test_a_query_that_is_nan_and_sees_nothing():
    c = Case([5], [2], 2, 1, 16, seed=52)
    c.q[0] = float("nan")
    out, lse = c.run()
    assert not out[:3].any() and torch.isneginf(lse[:3]).all()


@pytest.mark.parametrize("page", [16, 128])
def test_pages_given_up_are_hidden(page):
    c = Case([2, 150], [700, 700], 2, 1, page, seed=15)
    for col in (0, 2, 3):
        c.table[0][col] = -1
    c.table[1][1] = -5
    c.check()
    c.table[0] = [-1] * len(c.table[0])
    c.check()
    c.check(window=200, sinks=4)


def test_pages_past_the_cache_are_hidden_and_reported():
    c = Case([2, 1], [300, 40], 2, 1, 64, seed=16)
    n = c.k.shape[0]
    c.table[0][1], c.table[0][3] = n, 2**31 - 1
    result = c.run()
    assert kda.kda_device_status(clear=True) == INDEX
    c.check(result=result)
    c = Case([2, 1], [300, 40], 2, 1, 64, seed=16)
    c.table[0][0] = c.table[0][1] = n
    c.check(window=100)
    c.table[0][5] = n  # past the request's tokens
    c.check(window=100)


def test_lengths_outside_the_table():
    c = Case([2, 1, 1], [300, 40, 17], 2, 1, 64, seed=17, cols=5)
    real = list(c.kv)
    out, lse = kda.kda_paged_attention(c.cache(), c.q, _i32(c.cu), _i32([321, 40, -4]), _i32(c.table), return_lse=True)
    assert kda.kda_device_status(clear=True) == INDEX
    c.check(result=(out, lse), rows=[2], kv=real)
    assert not out[3].any() and torch.isneginf(lse[3]).all()
    c.kv = [320, 40, 17]  # clamped to the table's 5 pages
    c.check(result=(out, lse), rows=[0, 1, 2])


@pytest.mark.parametrize("cu", [[0, 2, 1, 4], [0, 2, 3, 5], [-1, 2, 3, 4], [0, 9, 3, 4]])
def test_bad_row_starts(cu):
    c = Case([2, 1, 1], [300, 40, 17], 2, 1, 64, seed=18)
    out = torch.full((6, 2, 128), 7.0, dtype=BF16, device="cuda")
    kda.kda_paged_attention(c.cache(), c.q, _i32(cu), _i32(c.kv), _i32(c.table), out=out[:4])
    assert kda.kda_device_status(clear=True) == INDEX
    assert (out[4:] == 7).all() and torch.isfinite(out).all()


def test_rows_of_no_request_and_guards():
    c = Case([2, 130, 4], [300, 140, 17], 2, 1, 64, seed=19)
    full = torch.full((136 + 9, 2, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((136 + 9, 2), 7.0, device="cuda")
    table = torch.full((3, 9), 10**6, dtype=torch.int32, device="cuda")
    table[:, :len(c.table[0])] = _i32(c.table)
    kda.kda_paged_attention(c.cache(), c.q, _i32(c.cu[:3]), _i32(c.kv[:2]), table[:2, :len(c.table[0])], out=full[:136],
                            lse=lse[:136])
    assert (full[132:] == 7).all() and (lse[132:] == 7).all() and not (full[:132] == 7).all(-1).any()
    c.check(result=(full[:136], lse[:136]), rows=slice(0, 132))


# --- how it is called ----------------------------------------------------------------

def test_one_workspace_for_calls_of_all_shapes_and_both_caches():
    ws = kda.paged_attention_workspace(tokens=1001, heads=8)
    cases = [Case([1], [9000], 4, 1, 64, seed=20), Case([1] * 40, list(range(3, 1203, 30)), 8, 2, 16, seed=21),
             Case([700, 1, 300], [900, 2000, 300], 2, 2, 64, FP16, seed=22), Case([3], [3], 1, 1, 16, seed=23)]
    first = [c.run(workspace=ws) for c in cases]
    wide = torch.randn(2, 40, 64, 2, 128, device="cuda").bfloat16()
    q = torch.randn(300, 4, 128, device="cuda").bfloat16()
    table = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    args = kda.KvCache(wide[0], wide[1]), q, _i32([0, 300]), _i32([2000]), table
    a, _ = kda.kda_paged_attention(*args, workspace=ws)
    again = [c.run(workspace=ws) for c in reversed(cases)][::-1]
    b, _ = kda.kda_paged_attention(*args)
    assert torch.equal(a, b)
    alone = [c.run() for c in cases]
    for c, a, b, d in zip(cases, first, again, alone):
        c.check(result=a)
        for x, y in ((a, b), (a, d)):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert not ws[:4096].any()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_workspace_holds_anything_past_its_first_bytes(dtype):
    """Blocks cut in parts, some of them without keys, over a workspace whose rest is all ones (a
    NaN in each of its types): the same bits as over zeros."""
    cases = [Case([1], [9000], 4, 1, 64, dtype, seed=24), Case([300, 2, 70, 129], [1, 0, 1, 400], 3, 3, 16, dtype, seed=25),
             Case([700, 1, 300], [2900, 2000, 100], 2, 2, 64, dtype, seed=26)]
    for c in cases:
        zeros = kda.paged_attention_workspace(tokens=1001, heads=9)
        zeros.zero_()
        ones = torch.full_like(zeros, 255)
        ones[:4096] = 0
        want, got = c.run(workspace=zeros), c.run(workspace=ones)
        c.check(result=got)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_other_stream_and_graph():
    c = Case([1, 2, 150], [800, 700, 300], 4, 2, 64, seed=24)
    want = c.run()
    cache, ws = c.cache(), kda.paged_attention_workspace(tokens=153, heads=4)
    cu, kv, table = _i32(c.cu), _i32(c.kv), _i32(c.table)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, lse = kda.kda_paged_attention(cache, c.q, cu, kv, table, workspace=ws, return_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(got, want[0]) and torch.equal(lse, want[1])
    out, lse = torch.empty_like(got), torch.empty_like(lse)
    q = c.q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_paged_attention(cache, q, cu, kv, table, workspace=ws, out=out, lse=lse)
    for lens in ([800, 700, 300], [5, 700, 222], [800, 1, 150]):
        kv.copy_(_i32(lens))
        q.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        c.kv, c.q = lens, q
        c.check(result=(out, lse))


def test_a_call_on_another_stream_makes_what_it_needs_there():
    c = Case([1, 2, 150], [9000, 700, 300], 4, 2, 64, seed=61)
    want = c.run()
    cache, args = c.cache(), [_i32(x) for x in (c.cu, c.kv, c.table)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kda.kda_paged_attention(cache, c.q, *args, return_lse=True, stream=s)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    got = [kda.kda_paged_attention(cache, c.q, *args, return_lse=True, stream=s) for _ in range(3)]
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_cache_past_32_bit_offsets():
    page, hkv = 256, 64
    n_pages = (1 << 32) // (page * hkv * 128) + 4
    k = torch.zeros(n_pages, page, hkv, 128, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = torch.ones(2, n_pages, hkv, page // 16, device="cuda")
    small = Case([2, 1], [500, 300], hkv, hkv, page, seed=25)
    used = sorted(p for row in small.table for p in row if p >= 0)
    high = {p: n_pages - 1 - i for i, p in enumerate(used)}
    for p, to in high.items():
        k[to], v[to] = small.k.view(torch.uint8)[p], small.v.view(torch.uint8)[p]
        ks[to], vs[to] = small.ks[p], small.vs[p]
    out, lse = kda.kda_paged_attention(kda.KvCache(k.view(F8), v.view(F8), ks, vs, dtype=BF16), small.q, _i32(small.cu),
                                       _i32(small.kv), _i32([[high.get(p, -1) for p in row] for row in small.table]), return_lse=True)
    small.check(result=(out, lse))


# --- mixtures and repetition ----------------------------------------------------------

@pytest.mark.parametrize("seed", range(8))
def test_mixed_batches(seed):
    r = np.random.default_rng(100 + seed)
    hkv = int(r.choice([1, 2, 3]))
    hq = hkv * int(r.choice([1, 2, 3, 5, 8, 16]))
    new, kv = [], []
    for _ in range(int(r.integers(3, 40))):
        n = int(r.choice([0, 1, 1, 2, 5, 8, 9, 17, 40, 65, 130, 200]))
        new.append(n)
        kv.append(int(max(0, n + r.choice([-3, 0, 0, 1, 60, 127, 500, 1500]))))
    c = Case(new, kv, hq, hkv, int(r.choice([16, 32, 64, 128, 256])), FP16 if seed % 2 else BF16,
             ["tokens", "heads", "pairs"][seed % 3], seed=seed)
    window, sinks = [(0, 0), (0, 0), (33, 1), (400, 130)][seed % 4]
    first = c.run(window, sinks)
    c.check(window, sinks, result=first)
    ws = kda.paged_attention_workspace(tokens=sum(new) + 1, heads=hq)
    for _ in range(20):
        again = c.run(window, sinks, workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert not ws[:4096].any()


@pytest.mark.parametrize("rows", [63, 64, 65, 100, 128])
def test_blocks_of_one_tile(rows):
    Case([rows] * 40, [400 + rows] * 40, 1, 1, 64, seed=rows).check()
    Case([rows // 4] * 20, [rows // 4 + 300] * 20, 4, 1, 16, FP16, seed=rows).check()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows", [64, 65, 128])
def test_many_blocks_of_one_tile(rows, dtype):
    r = np.random.default_rng(rows)
    kv = [int(rows // 2 + n) for n in r.integers(1, 400, 600)]
    c = Case([rows // 2] * 600, kv, 2, 1, 128, dtype, seed=rows)
    first = c.run()
    c.check(result=first)
    for _ in range(10):
        again = c.run()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kv,page", [(700, 16), (3000, 64), (6100, 128)])
def test_small_blocks_with_long_caches_before_large_ones(kv, page, dtype):
    """Blocks of few rows go to one stream; the other comes to the next block, with many
    rows, long before its keys and values do."""
    c = Case([1, 40, 2, 90] * 12, [kv, 300, kv + 90, 95] * 12, 4, 2, page, dtype, seed=page)
    first = c.run()
    c.check(result=first)
    for _ in range(10):
        again = c.run()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


# --- a serving step: turned, written, attended to, read back --------------------------

@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_steps_of_a_layer(dtype):
    """Prompt chunks, single tokens and a rejected draft through rope, append and
    attention; each step against the definition on what the cache stands for."""
    hq, hkv, page, n_req = 6, 2, 16, 4
    pages = kda.KvPages.empty(n_req, 40, 160, page)
    cache = kda.KvCache.empty(160, page, hkv, dtype=dtype, quantized=True)
    f = kda.rope_frequencies(64, 5e5, factor=4.0, original_context=128)
    rope = kda.Rope(f, layout="pairs")
    g = torch.Generator(device="cuda").manual_seed(3)
    c = Case([1], [1], hq, hkv, page, dtype)  # for its check
    for step, (new, keep) in enumerate([([100, 7, 0, 1], None), ([130, 1, 300, 1], None), ([4, 4, 4, 4], [231, 9, 300, 5]),
                                        ([1, 1, 1, 1], None)]):
        before = pages.kv_lens.tolist()
        cu, slots, lens = kda.kda_kv_extend(pages, _i32(new), sum(new))
        qkv = torch.randn(sum(new), hq + 2 * hkv, 128, generator=g, device="cuda").to(dtype)
        q, k, v = qkv.split((hq, hkv, hkv), 1)
        raw = _np(k)
        kda.kda_rope(rope, q, k, cu_seqlens=cu, kv_lens=lens, q_out=q, k_out=k)
        pos = [b + i for b, n in zip(before, new) for i in range(n)]
        off = np.abs(_np(k) - quant.rope(raw, pos, f.tolist(), "pairs"))
        assert off.max() <= torch.finfo(dtype).eps / 2 * 8 * 1.001
        kda.kda_kv_append(cache, k, v, slots)
        out, lse = kda.kda_paged_attention(cache, q, cu, lens, pages.block_table, return_lse=True)
        c.k, c.v, c.ks, c.vs, c.q = cache.k, cache.v, cache.k_scale, cache.v_scale, q
        c.cu, c.kv, c.table = cu.tolist(), lens.tolist(), pages.block_table.tolist()
        c.check(result=(out, lse))
        back = kda.kda_kv_read(cache, slots)
        rows = [(s // page, s % page) for s in slots.tolist()]
        for x, want in zip(back, c.numbers()):
            assert np.array_equal(_np(x), np.stack([want[p, r] for p, r in rows]))
        if keep:
            kda.kda_kv_truncate(pages, _i32(keep))
    assert kda.kda_device_status() == 0
