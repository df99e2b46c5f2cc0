"""What is measured of the paged key/value cache beside the recurrent states:

pages      pages for a step's new tokens (block tables, slot maps, row starts)
           taken from a free list, and handed back when the tokens are dropped
append     the step's keys and values written to their cache slots
attention  causal softmax attention of the step's tokens (one per request, a
           short window, a prompt chunk, or all of these in one batch) over
           the paged cache, in full or with a sliding window and a few first
           tokens that stay visible

Every case is a dict of plain values; ``lens_of`` turns it into the request
lengths.  With ``own`` false ``run`` computes the operators from elementary
torch operations in 32 bits, with ``own`` true it calls the package.
"""
import math
import random

import torch

own = False

D = 128  # head dimension
NEG = float("-inf")
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # a small serving batch that decodes: one new token each, latency bound
        {"name": "pages 16 requests", "op": "pages", "n_req": 16, "new_lo": 1, "new_hi": 1, "old_lo": 1,
         "old_hi": 2048, "page": 16, "cols": 160, "spare": 64, "lens_seed": 1},
        # speculative decoding of a large batch: windows of four tokens, all rolled back
        {"name": "pages 2048 requests window 4", "op": "pages", "n_req": 2048, "new_lo": 4, "new_hi": 4,
         "old_lo": 0, "old_hi": 8192, "page": 64, "cols": 136, "spare": 4096, "lens_seed": 2},
        # prompt chunks of ragged lengths; the free list ends before the batch does
        {"name": "pages 48 prompt chunks", "op": "pages", "n_req": 48, "new_lo": 1, "new_hi": 4096, "old_lo": 0,
         "old_hi": 8192, "page": 64, "cols": 200, "spare": 1400, "lens_seed": 3},
        # one decode step of 256 requests, token-major pages
        {"name": "append 256 tokens", "op": "append", "tokens": 256, "hkv": 8, "page": 64, "n_pages": 2048,
         "head_major": False, "dtype": "bf16", "padding": 3},
        # a packed prefill batch, head-major pages, keys and values cut from one projection
        {"name": "append 32768 tokens", "op": "append", "tokens": 32768, "hkv": 8, "page": 16, "n_pages": 4096,
         "head_major": True, "dtype": "fp16", "padding": 0},
        # one conversation: a single token against its cache, latency bound
        {"name": "decode 1 request", "op": "attention", "n_req": 1, "new_lo": 1, "new_hi": 1, "old_lo": 4095,
         "old_hi": 4095, "chunks": 0, "chunk_hi": 1, "hq": 32, "hkv": 8, "page": 64, "window": 0, "sinks": 0,
         "head_major": False, "dtype": "bf16", "lens_seed": 6},
        # the serving batch of 256 requests, ragged caches, memory bound
        {"name": "decode 256 requests", "op": "attention", "n_req": 256, "new_lo": 1, "new_hi": 1, "old_lo": 512,
         "old_hi": 8191, "chunks": 0, "chunk_hi": 1, "hq": 32, "hkv": 8, "page": 64, "window": 0, "sinks": 0,
         "head_major": False, "dtype": "bf16", "lens_seed": 7},
        # verify windows of up to four drafted tokens in a layer with a sliding window, one key head per query head
        {"name": "window verify 64 requests", "op": "attention", "n_req": 64, "new_lo": 1, "new_hi": 4, "old_lo": 0,
         "old_hi": 16000, "chunks": 0, "chunk_hi": 1, "hq": 16, "hkv": 16, "page": 16, "window": 1024, "sinks": 4,
         "head_major": True, "dtype": "fp16", "lens_seed": 8},
        # packed prompts of ragged lengths with nothing cached
        {"name": "prefill 8 prompts", "op": "attention", "n_req": 8, "new_lo": 97, "new_hi": 4096, "old_lo": 0,
         "old_hi": 0, "chunks": 8, "chunk_hi": 4096, "hq": 32, "hkv": 8, "page": 64, "window": 0, "sinks": 0,
         "head_major": False, "dtype": "bf16", "lens_seed": 9},
        # one chunk of a long prompt over what came before, compute bound
        {"name": "chunk 8192 over 24576", "op": "attention", "n_req": 1, "new_lo": 8192, "new_hi": 8192,
         "old_lo": 24576, "old_hi": 24576, "chunks": 1, "chunk_hi": 8192, "hq": 32, "hkv": 32, "page": 128,
         "window": 0, "sinks": 0, "head_major": False, "dtype": "bf16", "lens_seed": 10},
        # a whole prompt through a layer with a sliding window and first tokens that stay
        {"name": "window prefill 16001", "op": "attention", "n_req": 1, "new_lo": 16001, "new_hi": 16001,
         "old_lo": 0, "old_hi": 0, "chunks": 1, "chunk_hi": 16001, "hq": 16, "hkv": 2, "page": 32, "window": 1024,
         "sinks": 16, "head_major": False, "dtype": "fp16", "lens_seed": 11},
        # continuous batching: prompt chunks among decoding requests, three query heads to a key head
        {"name": "mixed batch 64 requests", "op": "attention", "n_req": 64, "new_lo": 1, "new_hi": 2, "old_lo": 1,
         "old_hi": 6000, "chunks": 4, "chunk_hi": 512, "hq": 24, "hkv": 8, "page": 64, "window": 2048, "sinks": 4,
         "head_major": False, "dtype": "bf16", "lens_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    seed = rng.randrange(1 << 20)
    op = rng.choice(["pages", "append", "attention", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    if op == "pages":
        n_req = _log_int(rng, 1, 2048)
        new_hi = _log_int(rng, 1, max(1, min(4096, 98304 // n_req)))
        old_hi = rng.choice([0, _log_int(rng, 1, 8192)])
        cols = -(-(old_hi + new_hi) // page) + rng.randint(0, 9)
        want = n_req * (-(-new_hi // page))
        return {"op": op, "n_req": n_req, "new_lo": 0, "new_hi": new_hi, "old_lo": 0, "old_hi": old_hi, "page": page,
                "cols": cols, "spare": max(1, int(want * rng.uniform(0.3, 1.2))), "lens_seed": seed}
    hkv = rng.choice([1, 2, 4, 8, 16])
    dtype = rng.choice(["bf16", "fp16"])
    head_major = rng.random() < 0.5
    if op == "append":
        tokens = _log_int(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "hkv": rng.choice([1, 2, 3, 5, 8]), "page": page,
                "n_pages": -(-tokens // page) + _log_int(rng, 1, 2048), "head_major": head_major, "dtype": dtype,
                "padding": rng.randint(0, tokens // 8)}
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 6, 8, 16) if g * hkv <= 32])
    window = rng.choice([0, 0, _log_int(rng, 32, 8192)])
    sinks = rng.choice([0, 1, 4, 128]) if window else 0
    kind = rng.choice(["decode", "verify", "chunk", "mixed"])
    c = {"op": op, "n_req": 1, "new_lo": 1, "new_hi": 1, "old_lo": 0, "old_hi": 0, "chunks": 0, "chunk_hi": 1,
         "hq": hq, "hkv": hkv, "page": page, "window": window, "sinks": sinks, "head_major": head_major,
         "dtype": dtype, "lens_seed": seed}
    if kind in ("decode", "verify"):
        c["n_req"] = _log_int(rng, 1, 256)
        c["old_hi"] = _log_int(rng, 16, min(32768, (1 << 21) * 8 // (hkv * c["n_req"])))
        c["new_hi"] = 1 if kind == "decode" else rng.randint(2, 8)
    elif kind == "chunk":
        c["n_req"] = c["chunks"] = rng.choice([1, 1, 2, 5])
        c["old_hi"] = rng.choice([0, _log_int(rng, 16, 24576)])
        c["chunk_hi"] = _log_int(rng, 64, min(8192, (1 << 32) // (c["n_req"] * hq * (c["old_hi"] + 8192))))
        c["new_lo"] = c["new_hi"] = c["chunk_hi"]
        c["new_lo"] = max(1, c["new_lo"] // 3)
    else:
        c["n_req"] = _log_int(rng, 4, 64)
        c["chunks"] = rng.randint(1, 3)
        c["old_hi"] = _log_int(rng, 16, 8192)
        c["chunk_hi"] = _log_int(rng, 17, 384)
        c["new_hi"] = 2
    return c


def lens_of(case):
    """(new tokens, cached tokens before them) of every request, from the case alone."""
    r = random.Random(case["lens_seed"])
    old = [r.randint(case["old_lo"], case["old_hi"]) for _ in range(case["n_req"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n_req"])]
    if case.get("chunks") and case["new_hi"] < case["chunk_hi"]:
        for b in r.sample(range(case["n_req"]), min(case["chunks"], case["n_req"])):
            new[b] = r.randint(max(1, case["chunk_hi"] // 2), case["chunk_hi"])
    return new, old


def _ceil(a, b):
    return -(-a // b)


# --- inputs ------------------------------------------------------------------

def _cache(case, n_pages, g):
    """k and v as [page, token, head, 128] views of what the allocator gave: token-major or head-major pages."""
    dt, p, h = DTYPES[case["dtype"]], case["page"], case["hkv"]
    shape = (n_pages, h, p, D) if case["head_major"] else (n_pages, p, h, D)
    kv = [torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g) for _ in range(2)]
    return [x.permute(0, 2, 1, 3) if case["head_major"] else x for x in kv]


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _handles(s):
    """What a program keeps from its set-up on: the page pool's and the cache's handles, the workspace."""
    import linear_attention_serving_fwd_gb300 as kda

    if s["case"]["op"] == "pages":
        s["pool"] = kda.KvPages(s["kv_lens"], s["table"], s["free_pages"], s["free_count"], s["case"]["page"])
        return
    s["cache"] = kda.KvCache(s["k_cache"], s["v_cache"])
    if s["case"]["op"] == "attention":
        s["workspace"] = kda.paged_attention_workspace("cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    s = {"case": case}
    if case["op"] == "pages":
        new, old = lens_of(case)
        p = case["page"]
        owned = [_ceil(n, p) for n in old]
        n_pages = sum(owned) + case["spare"]
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        first = torch.tensor([0] + owned).cumsum(0)[:-1].cuda()
        col = torch.arange(case["cols"], device="cuda")
        own_col = col[None] < torch.tensor(owned, device="cuda")[:, None]
        table = torch.where(own_col, order[(first[:, None] + col[None]).clamp(max=n_pages - 1)], -1)
        free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        free[:case["spare"]] = order[sum(owned):]
        s.update(kv_lens=_int32(old), old_lens=_int32(old), new_lens=_int32(new), table=table.to(torch.int32).contiguous(),
                 free_pages=free, free_count=_int32([case["spare"]]), tokens=sum(new))
    elif case["op"] == "append":
        t, h = case["tokens"], case["hkv"]
        s["k_cache"], s["v_cache"] = _cache(case, case["n_pages"], g)
        kv = torch.empty((t, 2 * h, D), dtype=DTYPES[case["dtype"]], device="cuda").normal_(generator=g)
        s["k"], s["v"] = kv[:, :h], kv[:, h:]  # bands of one projection
        slots = torch.randperm(_ceil(t, case["page"]), generator=g, device="cuda")  # the last page stays out of use
        slots = slots[:, None] * case["page"] + torch.arange(case["page"], device="cuda")
        slots = slots.reshape(-1)[:t].to(torch.int32)
        if case["padding"]:
            slots[torch.randperm(t, generator=g, device="cuda")[:case["padding"]]] = -1
        s["slots"] = slots
    else:
        new, old = lens_of(case)
        p, hq, hkv, dt = case["page"], case["hq"], case["hkv"], DTYPES[case["dtype"]]
        kv = [a + b for a, b in zip(new, old)]
        owned = [_ceil(n, p) for n in kv]
        n_pages = sum(owned) + 1
        s["k_cache"], s["v_cache"] = _cache(case, n_pages, g)
        order = torch.randperm(n_pages - 1, generator=g, device="cuda").to(torch.int32)
        first = torch.tensor([0] + owned).cumsum(0)[:-1].cuda()
        col = torch.arange(max(owned), device="cuda")
        own_col = col[None] < torch.tensor(owned, device="cuda")[:, None]
        table = torch.where(own_col, order[(first[:, None] + col[None]).clamp(max=n_pages - 2)], -1)
        # queries share a direction to which the prompt's first keys answer
        u = torch.empty((hkv, D), device="cuda").normal_(generator=g)
        q = torch.empty((sum(new), hq, D), device="cuda").normal_(generator=g)
        s["q"] = (q + u.repeat_interleave(hq // hkv, 0)).to(dt)
        start = table[:, 0].long()
        s["k_cache"][start, :4] += (0.5 * u).to(dt)
        s.update(cu_seqlens=torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda(), kv_lens=_int32(kv),
                 table=table.to(torch.int32).contiguous(), scale=D ** -0.5)
    if own:
        _handles(s)
    torch.cuda.synchronize()
    return s


# --- one pass ----------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import linear_attention_serving_fwd_gb300 as kda

        if op == "pages":
            cu, slots, lens = kda.kda_kv_extend(s["pool"], s["new_lens"], s["tokens"])
            kda.kda_kv_truncate(s["pool"], s["old_lens"])
            return {"cu_seqlens": cu, "slot_map": slots, "step_lens": lens, "kv_lens": s["kv_lens"],
                    "table": s["table"], "free_pages": s["free_pages"], "free_count": s["free_count"]}
        if op == "append":
            kda.kda_kv_append(s["cache"], s["k"], s["v"], s["slots"])
            return {"k": s["k_cache"], "v": s["v_cache"]}
        c = s["case"]
        out, lse = kda.kda_paged_attention(s["cache"], s["q"], s["cu_seqlens"], s["kv_lens"], s["table"],
                                           scale=s["scale"], window=c["window"], sinks=c["sinks"], return_lse=True,
                                           workspace=s["workspace"])
        return {"out": out, "lse": lse}
    return {"pages": _pages_plain, "append": _append_plain, "attention": _attention_plain}[op](s)


def _pages_plain(s):
    p, table, free, count = s["case"]["page"], s["table"], s["free_pages"], s["free_count"]
    lens, new = s["kv_lens"], s["new_lens"]
    cols = torch.arange(table.shape[1], device=table.device)
    # take: requests in order, each the pages that its last token needs, while the list lasts
    have, need = (lens + p - 1) // p, (lens + new + p - 1) // p
    add = need - have
    upto = add.cumsum(0)
    fits = (add == 0) | (upto <= count)
    step = torch.where(fits, lens + new, 0)
    taken = fits[:, None] & (cols >= have[:, None]) & (cols < need[:, None])
    at = count - 1 - ((upto - add)[:, None] + cols - have[:, None])
    table.copy_(torch.where(taken, free[at.clamp(0, free.numel() - 1)], table))
    left = count - torch.where(fits, add, 0).sum()
    grown = torch.where(fits, lens + new, lens)
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0).to(torch.int32)])
    t = torch.arange(s["tokens"], device=table.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = lens[b] + (t - cu[b])
    page = table[b, (pos // p).clamp(max=table.shape[1] - 1)]
    slots = torch.where(fits[b], page * p + pos % p, -1).to(torch.int32)
    # give back: the pages past the kept lengths, so that the list is as before they were taken
    keep = torch.minimum(grown, s["old_lens"])
    have, kept = (grown + p - 1) // p, (keep + p - 1) // p
    drop = have - kept
    after = drop.sum() - drop.cumsum(0)
    gone = (cols >= kept[:, None]) & (cols < have[:, None])
    to = torch.where(gone, left + after[:, None] + (have[:, None] - 1 - cols), free.numel())
    longer = torch.cat([free, free[:1]])
    longer.scatter_(0, to.reshape(-1).long(), table.reshape(-1))
    free.copy_(longer[:-1])
    table.masked_fill_(gone, -1)
    count.copy_(left + drop.sum())
    lens.copy_(keep)
    return {"cu_seqlens": cu, "slot_map": slots, "step_lens": step.to(torch.int32), "kv_lens": lens, "table": table,
            "free_pages": free, "free_count": count}


def _append_plain(s):
    p, slots = s["case"]["page"], s["slots"].long()
    page, row = slots // p, slots % p
    spare = s["k_cache"].shape[0] - 1  # out of use: takes what has no slot, and is put back
    page = torch.where(slots < 0, spare, page)
    row = torch.where(slots < 0, 0, row)
    keep = s["k_cache"][spare, 0].clone(), s["v_cache"][spare, 0].clone()
    s["k_cache"][page, row] = s["k"]
    s["v_cache"][page, row] = s["v"]
    s["k_cache"][spare, 0] = keep[0]
    s["v_cache"][spare, 0] = keep[1]
    return {"k": s["k_cache"], "v": s["v_cache"]}


def _attention_plain(s):
    c, q, cu, kv = s["case"], s["q"], s["cu_seqlens"], s["kv_lens"]
    new, _ = lens_of(c)
    b, hkv, t = c["n_req"], c["hkv"], q.shape[0]
    grp, most = c["hq"] // hkv, max(new)
    pages = s["table"].clamp(min=0)
    # [request, key head, key, 128] in 32 bits
    k = s["k_cache"][pages].flatten(1, 2).transpose(1, 2).float()
    v = s["v_cache"][pages].flatten(1, 2).transpose(1, 2).float()
    n = k.shape[2]
    i = torch.arange(most, device=q.device)
    rows = (cu[:-1, None] + i).clamp(max=t - 1)
    qp = q[rows].float().view(b, most, hkv, grp, D).permute(0, 2, 3, 1, 4).reshape(b, hkv, grp * most, D)
    x = torch.matmul(qp, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, grp, most, n)
    pos = (kv - (cu[1:] - cu[:-1]))[:, None] + i
    j = torch.arange(n, device=q.device)
    seen = (j <= pos[..., None]) & (j < kv[:, None, None])
    if c["window"]:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    x.masked_fill_(~seen[:, None, None], NEG)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == NEG, 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hkv, grp * most, n), v).view(b, hkv, grp, most, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (total.log() + top).squeeze(-1)
    tok = torch.arange(t, device=q.device)
    of = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    at = tok - cu[of]
    return {"out": o[of, :, :, at].reshape(t, c["hq"], D).to(q.dtype), "lse": lse[of, :, :, at].reshape(t, c["hq"])}


# --- what a pass cannot do without -------------------------------------------

def work(case):
    if case["op"] == "pages":
        new, old = lens_of(case)
        n, t, p, left = len(new), sum(new), case["page"], case["spare"]
        taken = 0
        for a, o in zip(new, old):
            add = _ceil(o + a, p) - _ceil(o, p)
            if add <= left:
                left -= add
                taken += add
            elif add:
                left = 0
        # lengths in, starts, lengths and slots out; each page number is read and written on both ways
        return {"bytes": 4 * (3 * n + 3 * n + t + 8 * taken), "flops": 0}
    if case["op"] == "append":
        rows = case["tokens"] - case["padding"]
        return {"bytes": rows * case["hkv"] * D * 2 * 2 * 2 + 4 * case["tokens"], "flops": 0}
    new, old = lens_of(case)
    w, sinks, hq, hkv = case["window"], case["sinks"], case["hq"], case["hkv"]
    keys = pairs = 0
    for a, o in zip(new, old):
        if not w:
            keys += o + a
            pairs += a * o + a * (a + 1) // 2
            continue
        lo = max(0, o + 1 - w)  # first key of the first token's window
        keys += (o + a - lo) + min(sinks, lo)
        for pos in range(o, o + a):
            lo = max(0, pos + 1 - w)
            pairs += pos + 1 - lo + min(sinks, lo)
    t = sum(new)
    pages = sum(_ceil(a + o, case["page"]) for a, o in zip(new, old))
    return {"bytes": keys * hkv * D * 2 * 2 + t * hq * (D * 2 * 2 + 4) + 4 * (2 * len(new) + pages),
            "flops": 4 * D * hq * pairs}


# --- the definition in 64 bits -----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return _pages_exact(s)
    if case["op"] == "append":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        flat = s["slots"].long()
        for cache, rows in ((k, s["k"]), (v, s["v"])):
            for i in range(case["page"]):  # the slots that are row i of their page
                at = (flat % case["page"] == i) & (flat >= 0)
                cache[flat[at] // case["page"], i] = rows[at].double()
        return {"k": k, "v": v}
    return _attention_exact(s)


def _pages_exact(s):
    p = s["case"]["page"]
    lens, new, table = s["kv_lens"].tolist(), s["new_lens"].tolist(), s["table"].tolist()
    free, count = s["free_pages"].tolist(), int(s["free_count"])
    old, stack = list(lens), free[:count]
    cu, slots, step, full = [0], [], [], False
    for b, n in enumerate(new):
        have, need = _ceil(lens[b], p), _ceil(lens[b] + n, p)
        full = full or need - have > len(stack)
        ok = need == have or not full
        if ok:
            for col in range(have, need):
                table[b][col] = stack.pop()
            lens[b] += n
        slots += [table[b][(old[b] + i) // p] * p + (old[b] + i) % p if ok else -1 for i in range(n)]
        step.append(lens[b] if ok else 0)
        cu.append(cu[-1] + n)
    for b in reversed(range(len(new))):
        for col in reversed(range(_ceil(old[b], p), _ceil(lens[b], p))):
            stack.append(table[b][col])
            table[b][col] = -1
    at = {"cu_seqlens": cu, "slot_map": slots, "step_lens": step, "kv_lens": old, "table": table,
          "free_pages": stack + free[len(stack):], "free_count": [len(stack)]}
    return {k: torch.tensor(x, dtype=torch.int32) for k, x in at.items()}


def _attention_exact(s):
    c, q = s["case"], s["q"]
    new, old = lens_of(c)
    grp, p = c["hq"] // c["hkv"], c["page"]
    if sum(a * (a + o) for a, o in zip(new, old)) * c["hq"] > 1 << 34:
        return None
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], NEG, dtype=torch.float64, device=q.device)
    at = 0
    for b, (a, o) in enumerate(zip(new, old)):
        n = a + o
        pages = s["table"][b, :_ceil(n, p)].long()
        pos = torch.arange(o, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        hidden = j > pos
        if c["window"]:
            hidden = hidden | ((j <= pos - c["window"]) & (j >= c["sinks"]))
        for h in range(c["hkv"]):
            k = s["k_cache"][pages, :, h].reshape(-1, D)[:n].double()
            v = s["v_cache"][pages, :, h].reshape(-1, D)[:n].double()
            for x in range(h * grp, (h + 1) * grp):
                w = (q[at:at + a, x].double() @ k.T) * s["scale"]
                w = torch.where(hidden, NEG, w)
                lse[at:at + a, x] = torch.logsumexp(w, -1)
                out[at:at + a, x] = torch.softmax(w, -1) @ v
        at += a
    return {"out": out, "lse": lse}
