"""Attention over the paged cache against the fp64 oracle.

Tolerance, element by element, with u = eps / 2 of the 16-bit type (half a
step, relative): the output is rounded to that type once (u |o|) and so is
each weight before the product with the values (u W, W = sum_j p_j |v_j|, the
normalised p).  In fp16 a weight may also fall below the normal range: at
most 2^-25 of the largest, per key (n 2^-25 max|v|).  The 32-bit steps: a
score is off by at most 128 additions at 2^-24 of sum |q_i k_i| scale, which
is below 128 * 2^-24 * 16 = 2^-13 here, so p is off by as much, and the sum
as well: 2^-12 W, and 2^-13 + 2^-22 |lse| for the lse.  Rows that see nothing
are exactly 0 and -inf."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from oracle import paged

pytestmark = pytest.mark.gpu
INDEX = 5
BF16, FP16 = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _np(x):
    return x.double().cpu().numpy()


class Case:
    """new, kv: tokens of each request and its cached tokens, these included."""

    def __init__(self, new, kv, hq, hkv, page, dtype=BF16, layout="tokens", seed=0, gain=1.0, extra_cols=1, cols=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
        owned = [-(-n // page) for n in kv]
        n_pages = sum(owned) + 2
        shape = (n_pages, hkv, page, 128) if layout == "heads" else (n_pages, page, hkv, 128)
        if layout == "pairs":
            both = rnd(n_pages, 2, page, hkv, 128)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = rnd(*shape), rnd(*shape)
            if layout == "heads":
                self.k, self.v = self.k.permute(0, 2, 1, 3), self.v.permute(0, 2, 1, 3)
        ids = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        cols = cols or max(owned + [1]) + extra_cols
        self.table = []
        for n in owned:
            self.table.append([ids.pop() for _ in range(n)] + [-1] * (cols - n))
        t = sum(new)
        self.q = (rnd(t, hq + 2, 128) * gain)[:, 1:hq + 1]  # a band of a wider projection
        self.cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.new, self.kv, self.page, self.dtype, self.scale = new, list(kv), page, dtype, 128 ** -0.5
        self.owned = owned

    def rows(self, b):
        """(page, row) of request b's tokens in order."""
        return [(self.table[b][j // self.page], j % self.page) for j in range(self.kv[b])]

    def run(self, window=0, sinks=0, **kw):
        out, lse = kda.kda_paged_attention(kda.KvCache(self.k, self.v), self.q, _i32(self.cu), _i32(self.kv),
                                           _i32(self.table), scale=self.scale, window=window, sinks=sinks,
                                           return_lse=True, **kw)
        return out, lse

    def check(self, window=0, sinks=0, result=None, rows=slice(None), q=None, k=None, v=None, kv=None):
        out, lse = self.run(window, sinks) if result is None else result
        want, want_lse, weight = paged.attention(
            _np(self.q if q is None else q), _np(self.k if k is None else k), _np(self.v if v is None else v), self.cu,
            self.kv if kv is None else kv, self.table, self.scale, window, sinks)
        out, lse = _np(out)[rows], _np(lse)[rows]
        want, want_lse, weight = want[rows], want_lse[rows], weight[rows]
        u = torch.finfo(self.dtype).eps / 2
        vmax = float(torch.nan_to_num(self.v.float(), 0, 0, 0).abs().max())
        tol = u * np.abs(want) + (u + 2.0 ** -12) * weight * (1 + u)
        tol += (max(self.kv + [0]) * 2.0 ** -25 * vmax if self.dtype == FP16 else 0) + 1e-30
        empty = np.isneginf(want_lse)
        assert np.array_equal(empty, np.isneginf(lse)) and not out[empty].any()
        off = np.abs(out - want) - tol
        assert np.isfinite(out).all() and off.max(initial=-1) <= 0, f"{np.argmax(off)}: {off.max()}"
        lse_off = np.abs(lse[~empty] - want_lse[~empty]) - 2.0 ** -13 - 2.0 ** -22 * np.abs(want_lse[~empty])
        assert lse_off.max(initial=-1) <= 0, lse_off.max()
        assert kda.kda_device_status() == 0


# --- lengths, heads, pages, windows ---------------------------------------------

@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 385, 1000])
@pytest.mark.parametrize("dtype,layout,page", [(BF16, "tokens", 16), (FP16, "heads", 64), (BF16, "pairs", 256)])
def test_single_tokens(kv, dtype, layout, page):
    Case([1, 1], [kv, max(1, kv - 1)], 4, 2, page, dtype, layout, seed=kv).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (10, 2), (6, 1), (7, 1), (8, 1), (24, 2), (16, 1), (33, 1),
                                   (128, 1), (100, 1)])
@pytest.mark.parametrize("new,kv", [([1, 3], [200, 130]), ([150], [150]), ([40], [300])])
def test_head_groups(hq, hkv, new, kv):
    Case(new, kv, hq, hkv, 32, seed=hq).check()


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
    Case(new, kv.tolist(), 4, 2, 32, seed=5).check(window=64, sinks=4)


def test_more_requests_than_a_block_counts():
    n = 3000
    Case([1] * n, [1 + i % 37 for i in range(n)], 1, 1, 16, seed=6).check()


@pytest.mark.parametrize("gain", [8.0, 40.0])
def test_sharp_scores(gain):
    """Rows whose maximum grows from tile to tile, and rows with one weight."""
    c = Case([3, 140], [900, 400], 2, 1, 64, seed=9, gain=gain)
    for b in range(2):
        for j, (page, row) in enumerate(c.rows(b)):
            c.k[page, row] *= 0.2 + j / 400
    # scores reach a few hundred here: the 32-bit bound scales with them
    out, lse = c.run()
    want, want_lse, weight = paged.attention(_np(c.q), _np(c.k), _np(c.v), c.cu, c.kv, c.table, c.scale)
    reach = float(np.abs(_np(c.q)).sum(-1).max() * np.abs(_np(c.k)).max() * c.scale)
    eps = 128 * 2.0 ** -24 * reach
    u = 2.0 ** -8
    assert (np.abs(_np(out) - want) <= u * np.abs(want) + (u + 2 * eps) * weight * (1 + u) + 1e-30).all()
    assert (np.abs(_np(lse) - want_lse) <= eps + 2.0 ** -22 * np.abs(want_lse)).all()


# --- rows that see nothing, hidden places ------------------------------------------

def test_rows_before_the_cache_begins():
    """More tokens than cached ones: the first stand before position 0."""
    Case([5, 200, 3], [2, 130, 0], 2, 1, 16, seed=11).check()
    Case([300], [1], 4, 2, 64, FP16, seed=12).check(window=7, sinks=2)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_hidden_places_have_no_influence(poison, page, window, sinks):
    c = Case([3, 140, 1], [50, 300, 413], 2, 1, page, seed=13)
    clean_k, clean_v = c.k.clone(), c.v.clone()
    used = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    for b in range(3):
        for j, (pg, row) in enumerate(c.rows(b)):
            first = c.kv[b] - c.new[b]
            lo = first + 1 - window if window else 0
            used[pg, row] = j >= lo or j < sinks
    c.k[~used], c.v[~used] = poison, poison
    c.check(window, sinks, k=clean_k, v=clean_v)


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_a_poisoned_token_reaches_the_rows_that_see_it_alone(poison):
    """The chunk's own tokens: key and value of one of them are not finite."""
    c = Case([200, 1], [260, 40], 2, 1, 32, seed=14)
    at = 60 + 77  # position of token 77
    pg, row = c.rows(0)[at]
    clean = c.k.clone(), c.v.clone()
    c.v[pg, row, 0, 5] = poison
    out, lse = c.run()
    c.check(result=(out, lse), rows=slice(0, 77), k=clean[0], v=clean[1])
    c.check(result=(out, lse), rows=slice(200, 201), k=clean[0], v=clean[1])
    assert not torch.isfinite(out[77:200, :, 5]).any() and torch.isfinite(lse[77:]).all()
    assert torch.isfinite(out[77:200, :, :5]).all() and torch.isfinite(out[77:200, :, 6:]).all()
    c.k[pg, row, 0, 9] = float("nan")
    out, lse = c.run()
    c.check(result=(out, lse), rows=slice(0, 77), k=clean[0], v=clean[1])
    assert torch.isnan(out[77:200]).all() and torch.isnan(lse[77:200]).all()
    c.k[pg, row, 0, 9] = clean[0][pg, row, 0, 9]
    # out of a window that begins after it, but inside its tile
    out, lse = c.run(window=30)
    seen = list(range(77)) + list(range(107, 201))
    c.check(window=30, result=(out, lse), rows=seen, k=clean[0], v=clean[1])


@pytest.mark.parametrize("page", [16, 128])
def test_pages_given_up_are_hidden(page):
    """Negative entries: pages that left a window, or were never there."""
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
    # out of sight they are not met
    c = Case([2, 1], [300, 40], 2, 1, 64, seed=16)
    c.table[0][0] = c.table[0][1] = n
    c.check(window=100)
    c.table[0][5] = n  # past the request's tokens
    c.check(window=100)


def test_lengths_outside_the_table():
    c = Case([2, 1, 1], [300, 40, 17], 2, 1, 64, seed=17, cols=5)
    real = list(c.kv)
    out, lse = kda.kda_paged_attention(kda.KvCache(c.k, c.v), c.q, _i32(c.cu), _i32([321, 40, -4]), _i32(c.table),
                                       return_lse=True)
    assert kda.kda_device_status(clear=True) == INDEX
    c.check(result=(out, lse), rows=[2], kv=real)
    assert not out[3].any() and torch.isneginf(lse[3]).all()
    # clamped to the table's 5 pages
    c.kv = [320, 40, 17]
    c.check(result=(out, lse), rows=[0, 1, 2])


@pytest.mark.parametrize("cu", [[0, 2, 1, 4], [0, 2, 3, 5], [-1, 2, 3, 4], [0, 9, 3, 4]])
def test_bad_row_starts(cu):
    c = Case([2, 1, 1], [300, 40, 17], 2, 1, 64, seed=18)
    out = torch.full((6, 2, 128), 7.0, dtype=BF16, device="cuda")
    kda.kda_paged_attention(kda.KvCache(c.k, c.v), c.q, _i32(cu), _i32(c.kv), _i32(c.table), out=out[:4])
    assert kda.kda_device_status(clear=True) == INDEX
    assert (out[4:] == 7).all() and torch.isfinite(out).all()


def test_rows_of_no_request_and_guards():
    c = Case([2, 130, 4], [300, 140, 17], 2, 1, 64, seed=19)
    full = torch.full((136 + 9, 2, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((136 + 9, 2), 7.0, device="cuda")
    table = torch.full((3, 9), 10**6, dtype=torch.int32, device="cuda")
    table[:, :len(c.table[0])] = _i32(c.table)
    kda.kda_paged_attention(kda.KvCache(c.k, c.v), c.q, _i32(c.cu[:3]), _i32(c.kv[:2]), table[:2, :len(c.table[0])],
                            out=full[:136], lse=lse[:136])
    assert (full[132:] == 7).all() and (lse[132:] == 7).all() and not (full[:132] == 7).all(-1).any()
    c.check(result=(full[:136], lse[:136]), rows=slice(0, 132))


# --- how it is called ----------------------------------------------------------------

def test_one_workspace_for_calls_of_all_shapes_and_the_same_bits_twice():
    ws = kda.paged_attention_workspace()
    cases = [Case([1], [9000], 4, 1, 64, seed=20), Case([1] * 40, list(range(3, 1203, 30)), 8, 2, 16, seed=21),
             Case([700, 1, 300], [900, 2000, 300], 2, 2, 64, FP16, seed=22), Case([3], [3], 1, 1, 16, seed=23)]
    first = [c.run(workspace=ws) for c in cases]
    again = [c.run(workspace=ws) for c in reversed(cases)][::-1]
    alone = [c.run() for c in cases]
    for c, a, b, d in zip(cases, first, again, alone):
        c.check(result=a)
        for x, y in ((a, b), (a, d)):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert not ws[:4096].any()


def test_other_stream_and_graph():
    c = Case([1, 2, 150], [800, 700, 300], 4, 2, 64, seed=24)
    want = c.run()
    cache, ws = kda.KvCache(c.k, c.v), kda.paged_attention_workspace()
    cu, kv, table = _i32(c.cu), _i32(c.kv), _i32(c.table)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, lse = kda.kda_paged_attention(cache, c.q, cu, kv, table, workspace=ws, return_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(got, want[0]) and torch.equal(lse, want[1])
    out, lse = torch.empty_like(got), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_paged_attention(cache, c.q, cu, kv, table, workspace=ws, out=out, lse=lse)
    for lens in ([800, 700, 300], [5, 700, 222], [800, 1, 150]):
        kv.copy_(_i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        c.kv = lens
        c.check(result=(out, lse))


def test_a_cache_past_32_bit_offsets():
    page, hkv = 256, 64
    n_pages = (1 << 31) // (page * hkv * 128) + 4
    k = torch.empty(n_pages, page, hkv, 128, dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    small = Case([2, 1], [500, 300], hkv, hkv, page, seed=25)
    used = sorted(p for row in small.table for p in row if p >= 0)
    high = {p: n_pages - 1 - i for i, p in enumerate(used)}
    for p, to in high.items():
        k[to], v[to] = small.k[p], small.v[p]
    out, lse = kda.kda_paged_attention(kda.KvCache(k, v), small.q, _i32(small.cu), _i32(small.kv),
                                       _i32([[high.get(p, -1) for p in row] for row in small.table]), return_lse=True)
    small.check(result=(out, lse))


def test_refusals():
    c = Case([2], [30], 2, 1, 16)
    cache = kda.KvCache(c.k, c.v)
    a = dict(q=c.q, cu_seqlens=_i32(c.cu), kv_lens=_i32(c.kv), block_table=_i32(c.table))
    for over, error in [(dict(q=c.q.half()), TypeError), (dict(q=c.q[..., :64]), ValueError),
                        (dict(cu_seqlens=_i32([0])), ValueError), (dict(kv_lens=_i32(c.kv).long()), TypeError),
                        (dict(block_table=_i32(c.table + c.table)), ValueError),
                        (dict(out=torch.empty(2, 2, 128, device="cuda")), ValueError),
                        (dict(lse=torch.empty(2, 3, device="cuda")), ValueError), (dict(scale=0.0), ValueError),
                        (dict(window=-1), ValueError), (dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                                                        ValueError)]:
        args = {**a, **over}
        with pytest.raises(error):
            kda.kda_paged_attention(cache, args.pop("q"), args.pop("cu_seqlens"), args.pop("kv_lens"),
                                    args.pop("block_table"), **args)
    with pytest.raises(ValueError):
        kda.kda_kv_append(cache, c.q[:, :1], c.q[:1, :1], _i32([0, 1]))


# --- mixtures and repetition: what the warps of a block hand to each other ------------

@pytest.mark.parametrize("seed", range(8))
def test_mixed_batches(seed):
    """Single tokens, short windows, chunks of one and of several blocks, empty
    requests and rows before the cache, in one call, groups of all kinds."""
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
    ws = kda.paged_attention_workspace()
    for _ in range(20):
        again = c.run(window, sinks, workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert not ws[:4096].any()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_scores_that_climb(dtype):
    """Each row's maximum grows by a little from key to key, by hundreds over the
    cache: the reference moves many times, in some rows of a warp and not in
    others."""
    c = Case([2, 150], [1500, 700], 2, 1, 64, dtype, seed=31)
    direction = torch.ones(128, device="cuda", dtype=dtype)
    c.q[::3] = direction  # every third token
    for b in range(2):
        for j, (page, row) in enumerate(c.rows(b)):
            c.k[page, row] = c.k[page, row] * 0.05 + j / 60
    out, lse = c.run()
    want, want_lse, weight = paged.attention(_np(c.q), _np(c.k), _np(c.v), c.cu, c.kv, c.table, c.scale)
    reach = float(np.abs(_np(c.q)).sum(-1).max() * np.abs(_np(c.k)).max() * c.scale)
    eps, u = 128 * 2.0 ** -24 * reach, torch.finfo(dtype).eps / 2
    small = 1500 * 2.0 ** -25 * float(c.v.float().abs().max()) if dtype == FP16 else 0.0
    assert (np.abs(_np(out) - want) <= u * np.abs(want) + (u + 2 * eps) * weight * (1 + u) + small + 1e-30).all()
    assert (np.abs(_np(lse) - want_lse) <= eps + 2.0 ** -22 * np.abs(want_lse)).all()


@pytest.mark.parametrize("rows", [63, 64, 65, 100, 128])
def test_blocks_of_one_tile(rows):
    """Blocks that fit one tile, up to all of its rows, one after another in a
    block's queue."""
    Case([rows] * 40, [400 + rows] * 40, 1, 1, 64, seed=rows).check()
    Case([rows // 4] * 20, [rows // 4 + 300] * 20, 4, 1, 16, FP16, seed=rows).check()


@pytest.mark.parametrize("rows", [64, 65, 128])
def test_many_blocks_of_one_tile(rows):
    """Several such blocks in each queue, of one key tile to four, so that either
    stream leads and blocks that join their streams' results follow one another."""
    r = np.random.default_rng(rows)
    kv = [int(rows // 2 + n) for n in r.integers(1, 400, 600)]
    c = Case([rows // 2] * 600, kv, 2, 1, 128, seed=rows)
    first = c.run()
    c.check(result=first)
    for _ in range(10):
        again = c.run()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("window", [2**31 - 1, 10**6, 321])
def test_windows_past_the_table(window):
    c = Case([200, 3], [130, 300], 2, 1, 64, seed=41)
    a, b = c.run(window=window, sinks=3), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(result=a)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kv", [65, 100, 128, 129])
def test_halves_of_a_tile_that_differ(kv, dtype):
    """One or two key tiles, whose last moves the reference, the larger scores in
    one half of the keys or in the other: both halves have to weigh against the
    same reference, time after time."""
    c = Case([1, 30, 2, 128] * 50, [kv] * 200, 2, 2, 32, dtype, seed=kv)
    c.q[..., :64] = 1.0  # 64 dimensions that set a key's score for all rows alike
    for b in range(200):
        rows = torch.tensor(c.rows(b), device="cuda")
        first_half = torch.arange(kv, device="cuda") % 128 < 64
        level = torch.where(first_half == (b % 3 == 0), 1.0, -1.0) * (1 + b % 5) / 8
        c.k[rows[:, 0], rows[:, 1], :, :64] = level[:, None, None].to(dtype)
    first = c.run()
    c.check(result=first)
    ws = kda.paged_attention_workspace()
    for _ in range(30):
        again = c.run(workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


# --- visible NaN, in blocks that several CTAs or both streams share ---------------------

def _nan_rows(c, bad, window=0, sinks=0):
    """Rows ``bad`` [T, Hq] are NaN throughout, the others as if nothing were."""
    out, lse = c.run(window, sinks)
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.isfinite(out[~bad]).all() and torch.isfinite(lse[~bad]).all()
    k, v, q = [torch.nan_to_num(x.float(), 0.0).double().cpu().numpy() for x in (c.k, c.v, c.q)]
    want, want_lse, _ = paged.attention(q, k, v, c.cu, c.kv, c.table, c.scale, window, sinks)
    clean = (torch.from_numpy(want).to(out), torch.from_numpy(want_lse).to(lse))
    out, lse = torch.where(bad[..., None], clean[0], out), torch.where(bad, clean[1], lse)
    c.check(window, sinks, result=(out, lse), q=torch.from_numpy(q), k=torch.from_numpy(k), v=torch.from_numpy(v))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("new,kv", [([1], [9000]), ([1], [200]), ([1, 3], [20000, 300]), ([3], [5]), ([160], [5000]),
                                    ([300, 1], [2600, 1]), ([20] * 40, [600] * 40)])
def test_a_query_that_is_nan(new, kv, dtype):
    c = Case(new, kv, 4, 2, 64, dtype, seed=51)
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[-1, 2] = bad[len(bad) // 2, 3] = True
    c.q[bad.nonzero(as_tuple=True)[0], bad.nonzero(as_tuple=True)[1], 17] = float("nan")
    _nan_rows(c, bad)
    _nan_rows(c, bad, window=500, sinks=4)


@pytest.mark.parametrize("new,kv,at", [([1, 1], [9000, 9000], (0, 1280)), ([1, 1], [9000, 300], (2000, 3300)),
                                       ([2, 40], [20000, 700], (17000, 20000)), ([1, 1], [256, 80], (128, 256)),
                                       ([1, 1], [256, 80], (0, 128)), ([140, 1], [4000, 90], (256, 1800))])
def test_a_run_of_keys_that_are_nan(new, kv, at):
    """All keys of several tiles, more than a part of a divided block: the rows of
    that request and key head are NaN, whatever the other parts hold."""
    c = Case(new, kv, 4, 2, 64, seed=52)
    rows = torch.tensor(c.rows(0)[at[0]:at[1]], device="cuda")
    c.k[rows[:, 0], rows[:, 1], 1] = float("nan")
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[:new[0], 2:] = True
    _nan_rows(c, bad)


def test_a_call_on_another_stream_makes_what_it_needs_there():
    """No workspace and no outputs given, the current stream busy: the call on the
    other stream waits for nothing of it, and finishes right."""
    c = Case([1, 2, 150], [9000, 700, 300], 4, 2, 64, seed=61)
    want = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    n = kda.paged_attention_workspace().numel()
    for stream in (torch.cuda.current_stream(), s):  # both pools hold blocks of the workspace's size that are not zero
        with torch.cuda.stream(stream):
            used = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
            del used
    pages = kda.KvPages.empty(2, 4, 8, 16)
    cache, args = kda.KvCache(c.k, c.v), [_i32(x) for x in (c.cu, c.kv, c.table, [5, 20])]
    lens = pages.kv_lens.clone()
    torch.cuda.synchronize()

    def calls():
        got = [kda.kda_paged_attention(cache, c.q, *args[:3], return_lse=True, stream=s) for _ in range(3)]
        return got, kda.kda_kv_extend(pages, args[3], 25, stream=s)

    calls()  # kernels are loaded and pools grown, which the current stream may have to wait for
    kda.kda_kv_truncate(pages, lens, stream=s)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    got, (cu, slots, step) = calls()
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert cu.tolist() == [0, 5, 25] and step.tolist() == [5, 20]
    assert slots.tolist() == list(range(5)) + list(range(16, 36))


# --- visible values that are not finite ------------------------------------------------

def _check_values(c, window=0, sinks=0, result=None):
    """Where the definition in 64 bits is NaN or infinite the result is the same;
    elsewhere (a value reaches its own dimension alone) it is as without such
    values."""
    out, lse = c.run(window, sinks) if result is None else result
    with np.errstate(invalid="ignore"):
        want, _, _ = paged.attention(_np(c.q), _np(c.k), _np(c.v), c.cu, c.kv, c.table, c.scale, window, sinks)
    clean = torch.nan_to_num(c.v.float(), 0.0, 0.0, 0.0)
    finite, _, _ = paged.attention(_np(c.q), _np(c.k), _np(clean), c.cu, c.kv, c.table, c.scale, window, sinks)
    bad = ~np.isfinite(want)
    np.testing.assert_array_equal(_np(out)[bad], want[bad])
    out = torch.where(torch.from_numpy(bad).cuda(), torch.from_numpy(finite).cuda(), out.double())
    c.check(window, sinks, result=(out, lse), v=clean)
    return bad


def _poison(c, b, head, marks):
    for at, dim, value in marks:
        page, row = c.rows(b)[at]
        c.v[page, row, head, dim] = float(value)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("new,kv", [([1, 1], [9000, 700]), ([2, 1], [300, 40]), ([150, 3], [700, 90]), ([300], [2600]),
                                    ([60] * 30, [500] * 30)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (250, 20)])
def test_visible_values_that_are_not_finite(new, kv, dtype, window, sinks):
    c = Case(new, kv, 4, 2, 64, dtype, seed=71)
    last = kv[0] - new[0]
    _poison(c, 0, 1, [(3, 5, "nan"), (4, 6, "inf"), (5, 7, "-inf"), (6, 8, "inf"), (7, 8, "-inf"), (last, 9, "nan"),
                      (last, 6, "inf"), (max(0, last - 200), 10, "inf"), (kv[0] - 1, 11, "nan"), (last + new[0] // 2, 12, "-inf")])
    _poison(c, len(kv) - 1, 0, [(kv[-1] - 1, slice(None), "nan")])
    assert _check_values(c, window, sinks).any()


def test_infinite_values_with_the_smallest_weights():
    """e^-40 of the largest: 0 in 16 bits, but not in the definition."""
    c = Case([1, 140], [1000, 700], 2, 1, 64, FP16, seed=72)
    c.q[...], c.k[...] = 1.0, 0.0
    for b in range(2):
        for j, (page, row) in enumerate(c.rows(b)):
            if j == 2:
                c.k[page, row] = -40 / 128 / c.scale
    _poison(c, 0, 0, [(2, 3, "inf"), (2, 4, "nan")])
    _poison(c, 1, 0, [(2, 3, "-inf"), (2, 4, "nan"), (600, 5, "inf")])
    bad = _check_values(c)
    assert bad[:, :, 3].all()


def test_large_values_under_a_reference_that_stands():
    """Weights that sum to thousands times values near the largest number."""
    c = Case([1, 130], [3000, 700], 2, 1, 64, BF16, seed=73)
    c.q[..., :64], c.q[..., 64:] = 1.0, 0.0
    for b in range(2):
        rows = torch.tensor(c.rows(b), device="cuda")
        c.k[rows[:, 0], rows[:, 1]] = torch.where(torch.arange(c.kv[b], device="cuda") < 128, 0.0, 1.0625).to(BF16)[:, None, None]
    c.v *= 1e36
    c.check()


def test_many_rows_of_a_long_cache_beside_others():
    """A chunk over 120,000 cached tokens in which one token's values are NaN: half
    of a tile's rows do not see it and are formed again, which takes long; nothing
    else does without its result."""
    n, kv, nan = 256, 120_000, 130
    c = Case([n, 2, 1], [kv, 500, 9000], 4, 1, 256, BF16, seed=74)
    _poison(c, 0, 0, [(kv - n + nan, slice(0, 64), "nan"), (70, 100, "inf"), (90, 101, "nan")])
    out, lse = c.run()
    assert kda.kda_device_status() == 0
    at = torch.tensor(c.rows(0), device="cuda")
    k, v = c.k[at[:, 0], at[:, 1], 0].double(), c.v[at[:, 0], at[:, 1], 0].double()
    clean, u = torch.nan_to_num(v, 0.0, 0.0, 0.0), torch.finfo(BF16).eps / 2
    for i in list(range(0, n, 16)) + [nan - 1, nan, n - 1]:
        end = kv - n + i + 1
        s = (c.q[i].double() @ k[:end].T) * c.scale
        w = torch.softmax(s, -1)
        want, weight = w @ clean[:end], w @ clean[:end].abs()
        want[:, 100], want[:, 101] = float("inf"), float("nan")
        if i >= nan:
            want[:, :64] = float("nan")
        fine = torch.isfinite(want)
        assert torch.equal(torch.isnan(out[i]), torch.isnan(want)) and torch.isinf(out[i, :, 100]).all()
        off = (out[i].double() - want).abs() - u * want.abs() - (u + 2.0 ** -12) * weight * (1 + u)
        assert off[fine].max() <= 0
        ref = torch.logsumexp(s, -1)
        assert ((lse[i].double() - ref).abs() <= 2.0 ** -13 + 2.0 ** -22 * ref.abs()).all()
    rest = slice(n, n + 3)
    c.cu, c.kv, c.table, c.q, c.k, c.v = [0, 2, 3], c.kv[1:], c.table[1:], c.q[rest], c.k, torch.nan_to_num(c.v, 0.0, 0.0, 0.0)
    c.check(result=(out[rest], lse[rest]))


def test_infinite_values_with_no_weight():
    """Scores of -inf: 0 times an infinite value is NaN where the row sees another
    key, before the first maximum and after it; a row that has only such scores
    is 0."""
    c = Case([4, 140], [40, 400], 2, 1, 64, BF16, seed=75)
    c.q[..., 0] = 1.0
    for b, at in ((0, list(range(36))), (1, [0, 1, 300])):
        for j in at:
            page, row = c.rows(b)[j]
            c.k[page, row, 0, 0] = -float("inf")
    _poison(c, 0, 0, [(3, 5, "inf"), (38, 6, "nan")])
    _poison(c, 1, 0, [(0, 7, "inf"), (300, 8, "-inf"), (300, 9, "nan"), (200, 10, "inf")])
    c.q[0, 1] = 0.0  # 0 times inf: this row's scores are NaN
    out, lse = c.run()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    c.q[0, 1, 0] = 1.0
    bad = _check_values(c)
    assert bad[:4, :, 5].all() and not bad[:, :, 0].any()
    c.kv[0] = 36  # request 0 sees scores of -inf alone
    out, lse = c.run()
    assert not out[:4].any() and torch.isneginf(lse[:4]).all()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (2, 100), (33, 0), (33, 130)])
@pytest.mark.parametrize("new,kv,hq,hkv", [([150, 3, 4], [700, 90, 9], 6, 3), ([129, 8], [129, 500], 16, 1)])
def test_rows_of_a_narrow_window_share_no_key(new, kv, hq, hkv, window, sinks):
    """A value that is not finite reaches the rows whose window holds it, and none
    beside them in their tile."""
    c = Case(new, kv, hq, hkv, 32, BF16, seed=76)
    for b in range(len(kv)):
        for i in range(0, new[b], 7):
            _poison(c, b, i % hkv, [(kv[b] - new[b] + i, slice(None) if i % 2 else 9, ("nan", "inf", "-inf")[i % 3])])
    assert _check_values(c, window, sinks).any()


@pytest.mark.parametrize("new,kv", [([3], [60]), ([2], [9000]), ([140, 1], [1500, 300])])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_rows_whose_scores_are_all_minus_infinity(new, kv, value):
    """Their sum is 0: out 0 and lse -inf, whatever the values that they see, and
    wherever their block is divided.  With one key more the values count."""
    c = Case(new, kv, 2, 1, 64, BF16, seed=77)
    c.q[..., 0] = 1.0
    rows = torch.tensor(c.rows(0), device="cuda")
    c.k[rows[:, 0], rows[:, 1], 0, 0] = -float("inf")
    _poison(c, 0, 0, [(1, slice(0, 40), value), (kv[0] // 2, 50, value), (kv[0] - new[0], 60, value)])
    out, lse = c.run()
    assert not out[:new[0]].any() and torch.isneginf(lse[:new[0]]).all()
    page, row = c.rows(0)[kv[0] - new[0] - 1]
    c.k[page, row, 0, 0] = 0.0
    _check_values(c)
