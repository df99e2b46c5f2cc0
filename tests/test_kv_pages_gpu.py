"""Pages taken, handed back and written to, against the oracle: whole numbers
and copies, so everything is equal bit for bit."""
from __future__ import annotations

import random

import pytest
import torch

import linear_attention_serving_fwd_gb300 as kda
from oracle import paged

pytestmark = pytest.mark.gpu
INDEX = 5


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """A pool on the GPU and the same one as lists."""

    def __init__(self, lens, page, cols, spare, seed=0, stride=None):
        owned = [-(-n // page) for n in lens]
        ids = list(range(sum(owned) + spare))
        random.Random(seed).shuffle(ids)
        self.page, self.lens, self.free, self.table = page, list(lens), ids[sum(owned):], []
        for n in owned:
            self.table.append([ids.pop(0) for _ in range(n)] + [-1] * (cols - n))
        n_pages = sum(owned) + spare
        full = torch.full((len(lens), stride or cols), -7, dtype=torch.int32, device="cuda")
        self.gpu_table = full[:, :cols]
        if lens:
            self.gpu_table.copy_(_i32(self.table))
        self.full = full
        self.gpu = kda.KvPages(_i32(lens), self.gpu_table, _i32(self.free + [-1] * (n_pages - spare)), _i32([spare]), page)

    def same(self):
        g = self.gpu
        assert g.kv_lens.tolist() == self.lens
        assert g.block_table.tolist() == self.table
        n = int(g.free_count)
        assert g.free_pages[:n].tolist() == self.free
        assert (self.full[:, self.gpu_table.shape[1]:] == -7).all()

    def extend(self, new, most=None):
        most = sum(new) if most is None else most
        cu, slots, step = paged.extend(self.lens, self.table, self.free, new, self.page)
        got = kda.kda_kv_extend(self.gpu, _i32(new), most)
        assert got[0].tolist() == cu and got[2].tolist() == step
        assert got[1].tolist() == (slots + [-1] * most)[:most]
        self.same()

    def truncate(self, keep):
        paged.truncate(self.lens, self.table, self.free, keep, self.page)
        kda.kda_kv_truncate(self.gpu, _i32(keep))
        self.same()


@pytest.mark.parametrize("n_req", [1, 2, 31, 33, 1023, 1024, 1025, 3000])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_steps_of_a_batch(n_req, page):
    r = random.Random(n_req * page)
    b = Both([r.choice([0, 1, page - 1, page, page + 1, r.randint(0, 5 * page)]) for _ in range(n_req)], page, 12,
             n_req * 4, seed=n_req, stride=13)
    for step in range(4):
        new = [r.choice([0, 1, 4, page, r.randint(0, 2 * page)]) for _ in range(n_req)]
        new = [min(x, 12 * page - y) for x, y in zip(new, b.lens)]
        before = list(b.lens)
        b.extend(new, most=sum(new) + (0, 1, 77, 5)[step])
        b.truncate([r.choice([x, y, (x + y) // 2, 0 if r.random() < 0.1 else y + 3]) for x, y in zip(before, b.lens)])
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("n_req,spare", [(40, 0), (40, 7), (40, 23), (2500, 1100), (2500, 1700)])
def test_the_free_list_ends_before_the_batch(n_req, spare):
    r = random.Random(spare)
    b = Both([r.randint(0, 64) for _ in range(n_req)], 16, 30, spare, seed=3)
    new = [r.choice([0, 1, 40, 300 if n_req < 100 else 2]) for _ in range(n_req)]
    before = list(b.lens)
    b.extend(new)
    b.truncate(before)
    assert kda.kda_device_status() == 0


def test_one_long_prompt():
    b = Both([5], 128, 1025, 1030)
    b.extend([131072])
    b.truncate([7])
    assert kda.kda_device_status() == 0


def test_truncate_undoes_extend():
    b = Both([17, 0, 300, 64], 64, 40, 99)
    state = [x.clone() for x in (b.gpu.kv_lens, b.gpu.block_table, b.gpu.free_pages, b.gpu.free_count)]
    lens = b.gpu.kv_lens.clone()
    kda.kda_kv_extend(b.gpu, _i32([1, 2000, 3, 64]), 2068)
    kda.kda_kv_truncate(b.gpu, lens)
    for x, y in zip(state, (b.gpu.kv_lens, b.gpu.block_table, b.gpu.free_pages, b.gpu.free_count)):
        assert torch.equal(x, y)


def test_no_requests():
    g = kda.KvPages.empty(0, 4, 8, 16)
    cu, slots, step = kda.kda_kv_extend(g, _i32([]), 3)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and step.numel() == 0
    kda.kda_kv_truncate(g, _i32([]))
    assert int(g.free_count) == 8


@pytest.mark.parametrize("lens,new,step", [
    ([3, 4], [-1, 2], [0, 6]),       # a negative length counts as no tokens
    ([-2, 4], [1, 2], [0, 6]),       # lengths outside the row
    ([65, 4], [1, 2], [0, 6]),
    ([60, 4], [5, 2], [0, 6]),       # more than the row holds
    ([60, 4], [2**31 - 1, 0], [0, 4]),
])
def test_bad_lengths_are_reported_and_not_admitted(lens, new, step):
    g = kda.KvPages.empty(2, 4, 16, 16)
    g.kv_lens.copy_(_i32(lens))
    g.block_table[1, 0] = 2
    g.block_table[0, :] = _i32([3, 4, 5, 6])
    _, slots, got = kda.kda_kv_extend(g, _i32(new), 8)
    assert got.tolist() == step and kda.kda_device_status(clear=True) == INDEX
    assert g.kv_lens.tolist() == [lens[0], step[1]] and int(g.free_count) == 16
    want = ([-1] * min(8, max(0, new[0])) + [2 * 16 + 4 + i for i in range(new[1])])[:8]
    assert slots.tolist() == want + [-1] * (8 - len(want))


def test_more_tokens_than_the_slot_map():
    g = kda.KvPages.empty(2, 4, 16, 16)
    guard = torch.full((12,), -9, dtype=torch.int32, device="cuda")
    cu, slots, step = kda.kda_kv_extend(g, _i32([5, 6]), 8, slot_map=guard[:8])
    assert cu.tolist() == [0, 5, 11] and kda.kda_device_status(clear=True) == INDEX
    assert slots.tolist() == [0, 1, 2, 3, 4, 16, 17, 18] and guard[8:].tolist() == [-9] * 4


@pytest.mark.parametrize("count,left", [(-3, 0), (17, 15)])
def test_a_bad_free_count(count, left):
    g = kda.KvPages.empty(1, 4, 16, 16)
    g.free_count.fill_(count)
    _, _, step = kda.kda_kv_extend(g, _i32([3]), 3)
    assert kda.kda_device_status(clear=True) == INDEX
    assert int(g.free_count) == left and step.tolist() == [3 if left else 0]


def test_a_bad_page_in_the_free_list():
    g = kda.KvPages.empty(1, 4, 16, 16)
    g.free_pages.fill_(16)
    _, slots, _ = kda.kda_kv_extend(g, _i32([3]), 3)
    assert kda.kda_device_status(clear=True) == INDEX and slots.tolist() == [-1] * 3


def test_bad_truncations():
    b = Both([20, 30], 16, 4, 0)
    kda.kda_kv_truncate(b.gpu, _i32([-1, 16]))
    assert kda.kda_device_status(clear=True) == INDEX
    assert b.gpu.kv_lens.tolist() == [20, 16] and int(b.gpu.free_count) == 1
    b.gpu.free_count.fill_(3)  # one place left of four
    kda.kda_kv_truncate(b.gpu, _i32([0, 0]))
    assert kda.kda_device_status(clear=True) == INDEX and int(b.gpu.free_count) == 4
    b.gpu.kv_lens.copy_(_i32([100, 16]))
    kda.kda_kv_truncate(b.gpu, _i32([0, 16]))
    assert kda.kda_device_status(clear=True) == INDEX and b.gpu.kv_lens.tolist() == [100, 16]


def _give_up(b, at):
    """The pages of columns ``at`` [(request, column)] back onto the stack by hand,
    negative entries in their place."""
    g = b.gpu
    for i, (r, col) in enumerate(at):
        n = len(b.free)
        g.free_pages[n], g.block_table[r, col] = b.table[r][col], -1 - i
        b.free.append(b.table[r][col])
        b.table[r][col] = -1 - i
    g.free_count.fill_(len(b.free))


@pytest.mark.parametrize("lens,cols,at", [
    ([40, 33], 4, [(0, 0), (1, 1)]),
    ([700, 64, 1], 60, [(0, c) for c in range(0, 43)] + [(1, 3)]),
    ([17000, 5, 20000], 1300, [(0, c) for c in range(0, 1062, 3)] + [(2, c) for c in range(1100)]),  # several rounds
    ([33] * 1500, 4, [(r, 1) for r in range(0, 1500, 7)]),
])
def test_pages_given_up_are_not_handed_back(lens, cols, at):
    b = Both(lens, 16, cols, 9, seed=7)
    _give_up(b, at)
    b.truncate([n // 2 if i % 2 else 0 for i, n in enumerate(lens)])
    assert kda.kda_device_status() == 0
    b.extend([min(300, 16 * cols - n) if i < 3 else 0 for i, n in enumerate(b.lens)])
    b.truncate([0] * len(lens))
    assert kda.kda_device_status() == 0 and sorted(b.free) == list(range(len(b.free)))
    assert int(b.gpu.free_count) == b.gpu.free_pages.numel()  # all of them, each once


def test_entries_past_the_cache_are_not_handed_back():
    b = Both([40, 33], 16, 4, 1)
    n = b.gpu.free_pages.numel()
    for r, col, bad in ((0, 1, n), (1, 0, 2**31 - 1)):
        b.table[r][col] = bad
        b.gpu.block_table[r, col] = bad
    free = list(b.free)
    paged.truncate(b.lens, b.table, b.free, [0, 0], 16, n_pages=n)
    kda.kda_kv_truncate(b.gpu, _i32([0, 0]))
    assert kda.kda_device_status(clear=True) == INDEX and len(b.free) == len(free) + 4
    b.same()


def test_a_batch_that_asks_for_more_pages_than_32_bits_count():
    n, cols = 48, (1 << 27) - 1
    table = torch.empty(n, cols, dtype=torch.int32, device="cuda")  # rows of 2^31 tokens: 26 GB
    table[:, :4] = -1
    g = kda.KvPages(_i32([0] * n), table, _i32(list(range(31, -1, -1))), _i32([32]), 16)
    new = [20, 5] + [2**31 - 20] * (n - 2)
    cu, slots, step = kda.kda_kv_extend(g, _i32(new), 25)
    assert kda.kda_device_status(clear=True) == INDEX  # more tokens than the slot map
    assert step.tolist() == [20, 5] + [0] * (n - 2) and int(g.free_count) == 29
    assert table[:3, :3].tolist() == [[0, 1, -1], [2, -1, -1], [-1, -1, -1]]
    assert slots.tolist() == list(range(20)) + list(range(32, 37))


# --- append --------------------------------------------------------------------

def _caches(layout, n_pages, page, hkv, dtype):
    if layout == "tokens":
        kv = torch.randn(2, n_pages, page, hkv, 128, device="cuda").to(dtype)
        return kv, kv[0], kv[1]
    if layout == "heads":
        kv = torch.randn(2, n_pages, hkv, page, 128, device="cuda").to(dtype)
        return kv, kv[0].permute(0, 2, 1, 3), kv[1].permute(0, 2, 1, 3)
    kv = torch.randn(n_pages, 2, page, hkv, 136, device="cuda").to(dtype)  # pairs in a page, padded rows
    return kv, kv[:, 0, ..., :128], kv[:, 1, ..., :128]


@pytest.mark.parametrize("layout", ["tokens", "heads", "pairs"])
@pytest.mark.parametrize("t,hkv,page,dtype", [(1, 1, 16, torch.bfloat16), (5, 3, 32, torch.float16),
                                             (257, 8, 64, torch.bfloat16), (4099, 2, 256, torch.float16)])
def test_append(layout, t, hkv, page, dtype):
    n_pages = -(-t // page) + 3
    _, k_cache, v_cache = _caches(layout, n_pages, page, hkv, dtype)
    kv = torch.randn(t, 2 * hkv + 1, 128, device="cuda").to(dtype)
    k, v = kv[:, :hkv], kv[:, hkv:2 * hkv]
    if t == 5:
        k = k[:, :1].expand(t, hkv, 128)  # one key head for all
    k[0, 0, 3] = float("nan")
    slots = torch.randperm(n_pages * page, device="cuda")[:t].to(torch.int32)
    slots[::3] = -1 if t > 1 else int(slots[0])
    want_k, want_v = k_cache.clone(), v_cache.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // page, s % page], want_v[s // page, s % page] = k[i], v[i]
    kda.kda_kv_append(kda.KvCache(k_cache, v_cache), k, v, slots)
    bits = lambda x: x.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(k_cache), bits(want_k)) and torch.equal(bits(v_cache), bits(want_v))
    assert kda.kda_device_status() == 0


def test_append_reports_slots_past_the_cache():
    _, k_cache, v_cache = _caches("tokens", 4, 16, 2, torch.bfloat16)
    before = k_cache.clone(), v_cache.clone()
    k = torch.randn(3, 2, 128, device="cuda").bfloat16()
    kda.kda_kv_append(kda.KvCache(k_cache, v_cache), k, k, _i32([64, 2**31 - 1, 63]))
    assert kda.kda_device_status(clear=True) == INDEX
    assert torch.equal(k_cache[3, 15], k[2]) and torch.equal(v_cache[3, 15], k[2])
    k_cache[3, 15], v_cache[3, 15] = before[0][3, 15], before[1][3, 15]
    assert torch.equal(k_cache, before[0]) and torch.equal(v_cache, before[1])


def test_append_past_32_bit_offsets():
    page, hkv = 256, 64
    n_pages = (1 << 31) // (page * hkv * 128) + 2
    k_cache = torch.empty(n_pages, page, hkv, 128, dtype=torch.bfloat16, device="cuda")
    v_cache = torch.empty_like(k_cache)
    k_cache[[0, 1, n_pages - 1]], v_cache[[0, 1, n_pages - 1]] = 0, 0
    k, v = torch.randn(2, 2, hkv, 128, device="cuda").bfloat16()
    kda.kda_kv_append(kda.KvCache(k_cache, v_cache), k, v, _i32([n_pages * page - 1, (n_pages - 1) * page]))
    assert torch.equal(k_cache[-1, -1], k[0]) and torch.equal(v_cache[-1, 0], v[1])
    assert not k_cache[:2].any() and not v_cache[:2].any() and kda.kda_device_status() == 0
