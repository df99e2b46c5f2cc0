"""Pins of the paged cache's oracle: closed forms and invariances."""
from __future__ import annotations

import numpy as np

from oracle import paged


def _case(kv, n, hq, hkv, page, seed=0):
    r = np.random.default_rng(seed)
    n_pages = -(-kv // page) + 2
    table = [list(r.permutation(n_pages)[:-(-kv // page)])]
    kc, vc = r.standard_normal((2, n_pages, page, hkv, 128))
    return r.standard_normal((n, hq, 128)), kc, vc, [0, n], [kv], table


def test_one_key_returns_its_value():
    q, kc, vc, cu, kv, table = _case(1, 1, 2, 1, 16)
    out, lse, _ = paged.attention(q, kc, vc, cu, kv, table, 0.1)
    np.testing.assert_allclose(out[0, 1], vc[table[0][0], 0, 0])
    np.testing.assert_allclose(lse[0], 0.1 * q[0] @ kc[table[0][0], 0, 0])


def test_equal_scores_average_the_visible_values():
    q, kc, vc, cu, kv, table = _case(40, 3, 1, 1, 16)
    values = vc[table[0]].reshape(-1, 1, 128)[:40, 0]
    out, lse, _ = paged.attention(0 * q, kc, vc, cu, kv, table, 1.0, window=8, sinks=2)
    for i, p in enumerate((37, 38, 39)):
        seen = [0, 1] + list(range(p - 7, p + 1))
        np.testing.assert_allclose(out[i, 0], values[seen].mean(0))
        np.testing.assert_allclose(lse[i, 0], np.log(10))


def test_window_of_the_whole_cache_is_no_window():
    case = _case(50, 7, 4, 2, 16)
    a = paged.attention(*case, 0.09)
    b = paged.attention(*case, 0.09, window=50)
    c = paged.attention(*case, 0.09, window=10, sinks=50)
    for x, y, z in zip(a, b, c):
        np.testing.assert_array_equal(x, y)
        np.testing.assert_array_equal(x, z)


def test_grouped_heads_equal_repeated_key_heads():
    q, kc, vc, cu, kv, table = _case(33, 5, 6, 2, 16)
    a = paged.attention(q, kc, vc, cu, kv, table, 0.09)[0]
    b = paged.attention(q, kc.repeat(3, 2), vc.repeat(3, 2), cu, kv, table, 0.09)[0]
    np.testing.assert_allclose(a, b)


def test_two_parts_join_by_their_lse():
    q, kc, vc, cu, kv, table = _case(64, 1, 1, 1, 16)
    whole, total, _ = paged.attention(q, kc, vc, cu, kv, table, 0.09)
    parts = [paged.attention(q, kc, vc, cu, kv, [[x if keep(i) else -1 for i, x in enumerate(table[0])]], 0.09)
             for keep in (lambda i: i < 1, lambda i: i >= 1)]
    w = [np.exp(lse - total)[..., None] for _, lse, _ in parts]
    np.testing.assert_allclose(whole, sum(a * o[0] for a, o in zip(w, parts)))


def test_nothing_visible():
    q, kc, vc, cu, kv, table = _case(2, 4, 1, 1, 16)
    out, lse, _ = paged.attention(q, kc, vc, cu, kv, table, 0.09)
    assert not out[:2].any() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()


def test_pages_are_taken_in_order_and_truncate_undoes_it():
    lens, table, free = [3, 16, 0], [[7, -1, -1], [5, -1, -1], [-1, -1, -1]], [9, 8, 6, 4]
    before = [list(x) for x in ([lens] + table + [free])]
    cu, slots, step = paged.extend(lens, table, free, [2, 17, 1], 16)
    assert cu == [0, 2, 19, 20] and step == [5, 33, 1] and table == [[7, -1, -1], [5, 4, 6], [8, -1, -1]]
    assert slots == [7 * 16 + 3, 7 * 16 + 4] + list(range(64, 80)) + [96, 128] and free == [9]
    paged.truncate(lens, table, free, [3, 16, 0], 16)
    assert [lens] + table + [free] == before


def test_the_first_request_without_pages_ends_the_admission():
    lens, table, free = [16, 15, 0, 0], [[1, -1], [2, -1], [-1, -1], [-1, -1]], [3]
    cu, slots, step = paged.extend(lens, table, free, [20, 1, 0, 1], 16)
    assert step == [0, 16, 0, 0] and slots == [-1] * 20 + [2 * 16 + 15, -1] and free == [3] and cu[-1] == 22


def test_pages_given_up_are_not_handed_back():
    lens, table, free = [40, 33], [[7, 3, 5, -1], [1, 2, 9, -1]], [4]
    table[0][0], free = -1, free + [7]  # left a window: the caller has handed it back
    table[1][1] = 12                    # no page of a cache of ten
    paged.truncate(lens, table, free, [0, 1], 16, n_pages=10)
    assert lens == [0, 1] and table == [[-1] * 4, [1, -1, -1, -1]] and free == [4, 7, 9, 5, 3]
    _, slots, _ = paged.extend(lens, table, free, [17, 0], 16)
    assert slots == list(range(48, 64)) + [80] and free == [4, 7, 9]
