"""The paged key/value cache's operators written out: page bookkeeping on
Python lists, attention in numpy fp64 from its definition."""
from __future__ import annotations

import numpy as np


def extend(kv_lens, table, free, new_lens, page):
    """Lists, updated in place (``free``: the stack of free pages).  Returns
    (cu_seqlens, slot_map, step_lens)."""
    cu, slots, step, full = [0], [], [], False
    for b, n in enumerate(new_lens):
        have, need = -(-kv_lens[b] // page), -(-(kv_lens[b] + n) // page)
        full = full or need - have > len(free)
        if need > have and full:
            slots += [-1] * n
            step.append(0)
        else:
            for col in range(have, need):
                table[b][col] = free.pop()
            slots += [table[b][p // page] * page + p % page for p in range(kv_lens[b], kv_lens[b] + n)]
            kv_lens[b] += n
            step.append(kv_lens[b])
        cu.append(cu[-1] + n)
    return cu, slots, step


def truncate(kv_lens, table, free, keep_lens, page, n_pages=None):
    """Entries that are no page (negative, or ``n_pages`` and above) are not
    handed back."""
    for b in reversed(range(len(kv_lens))):
        keep = min(keep_lens[b], kv_lens[b])
        for col in reversed(range(-(-keep // page), -(-kv_lens[b] // page))):
            if table[b][col] >= 0 and (n_pages is None or table[b][col] < n_pages):
                free.append(table[b][col])
            table[b][col] = -1
        kv_lens[b] = keep


def attention(q, k_cache, v_cache, cu_seqlens, kv_lens, table, scale, window=0, sinks=0):
    """q [T, Hq, 128], caches [pages, page, Hkv, 128] (fp64 arrays).  Returns
    (out [T, Hq, 128], lse [T, Hq], weight): ``weight`` = sum_j p_j |v_j| with
    the normalised p, the scale that rounding errors of p and v act on.  Rows
    of no request stay NaN."""
    t_total, hq, d = q.shape
    page, hkv = k_cache.shape[1], k_cache.shape[2]
    out, weight = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full((t_total, hq), np.nan)
    for b, kv in enumerate(kv_lens):
        t0, t1 = cu_seqlens[b], cu_seqlens[b + 1]
        j = np.arange(kv)
        pages = np.asarray([table[b][x // page] for x in range(0, kv, page)], dtype=np.int64)
        held = np.repeat((pages >= 0) & (pages < k_cache.shape[0]), page)[:kv]
        for i in range(t0, t1):
            p = kv - (t1 - t0) + i - t0
            seen = (j <= p) & held
            if window:
                seen &= (j > p - window) | (j < sinks)
            at = j[seen]
            for h in range(hq):
                if not at.size:
                    out[i, h], weight[i, h], lse[i, h] = 0.0, 0.0, -np.inf
                    continue
                g = h // (hq // hkv)
                k, v = k_cache[pages[at // page], at % page, g], v_cache[pages[at // page], at % page, g]
                s = scale * (k @ q[i, h])
                e = np.exp(s - s.max())
                out[i, h], weight[i, h] = e @ v / e.sum(), e @ np.abs(v) / e.sum()
                lse[i, h] = s.max() + np.log(e.sum())
    return out, lse, weight
