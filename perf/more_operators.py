"""What is measured of the softmax-attention layers' rotary positions and of the
paged key/value cache held in 8 bits:

rope       queries and keys of a step's tokens rotated by their positions, in
           either pairing, the whole head or its first part, frequencies as
           they are or scaled for long contexts
append     the step's keys and values written to their slots in 8 bits, with a
           scale for each block of 16 tokens and head that grows with them
read       cached tokens read back in 16 bits
attention  causal softmax attention of the step's tokens over the cache (one
           per request, a short window, a prompt chunk, or all of these in one
           batch), in full or with a sliding window and a few first tokens
           that stay visible

Every case is a dict of plain values; ``lens_of`` turns it into the request
lengths.  With ``own`` false ``run`` computes the operators from elementary
torch operations in 32 bits, with ``own`` true it calls the package.
"""
import math
import random

import torch

own = False

D = 128  # head dimension
BLOCK = 16  # tokens that share a scale
TOP, LEAST, MOST = 448.0, -48, 48  # largest 8-bit value; exponents of the scales
NEG = float("-inf")
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn


# --- cases -------------------------------------------------------------------

def _rope(name, n_req, new_lo, new_hi, old_hi, seed, **kw):
    return {"name": name, "op": "rope", "n_req": n_req, "new_lo": new_lo, "new_hi": new_hi, "old_lo": 0, "old_hi": old_hi,
            "lens_seed": seed, **kw}


def _kv(name, op, n_req, new_lo, new_hi, old_lo, old_hi, seed, **kw):
    return {"name": name, "op": op, "n_req": n_req, "new_lo": new_lo, "new_hi": new_hi, "old_lo": old_lo, "old_hi": old_hi,
            "chunks": 0, "chunk_hi": 1, "window": 0, "sinks": 0, "lens_seed": seed, **kw}


def listed():
    return [
        # one decode step of a small batch, latency bound
        _rope("rope 16 tokens", 16, 1, 1, 8192, 1, hq=32, hkv=8, layout="half", rot=128, base=10000.0, factor=1.0, original=0,
              dtype="bf16"),
        # packed prompts, pairs side by side in the first half of the head, frequencies scaled for positions far out
        _rope("rope 32768 tokens", 12, 1, 5500, 120000, 2, hq=32, hkv=8, layout="pairs", rot=64, base=500000.0, factor=8.0,
              original=8192, dtype="fp16"),
        # one decode step of 256 requests: most tokens land inside a block that holds others
        _kv("append 256 tokens", "append", 256, 1, 1, 0, 500, 3, hkv=8, page=64, head_major=False, dtype="bf16"),
        # a packed prefill batch of ragged prompts, head-major pages, keys and values cut from one projection
        _kv("append 32768 tokens", "append", 16, 1, 4096, 0, 40, 4, hkv=8, page=16, head_major=True, dtype="fp16"),
        # the prefix of one conversation, read back
        _kv("read 1000 tokens", "read", 1, 1000, 1000, 0, 0, 5, hkv=8, page=64, head_major=False, dtype="bf16"),
        # a batch of requests that moves to another pool
        _kv("read 65536 tokens", "read", 24, 1, 5400, 0, 0, 6, hkv=8, page=32, head_major=True, dtype="fp16"),
        # one conversation: a single token against its cache, latency bound
        _kv("decode 1 request", "attention", 1, 1, 1, 4095, 4095, 7, hq=32, hkv=8, page=64, head_major=False, dtype="bf16"),
        # the serving batch of 256 requests, ragged caches, memory bound
        _kv("decode 256 requests", "attention", 256, 1, 1, 512, 8191, 8, hq=32, hkv=8, page=64, head_major=False, dtype="bf16"),
        # verify windows of up to four drafted tokens in a layer with a sliding window, one key head per query head
        _kv("window verify 64 requests", "attention", 64, 1, 4, 0, 16000, 9, hq=16, hkv=16, page=16, head_major=True,
            dtype="fp16", **{"window": 1024, "sinks": 4}),
        # packed prompts of ragged lengths with nothing cached
        _kv("prefill 8 prompts", "attention", 8, 97, 4096, 0, 0, 10, hq=32, hkv=8, page=64, head_major=False, dtype="bf16"),
        # one chunk of a long prompt over what came before, compute bound
        _kv("chunk 8192 over 16384", "attention", 1, 8192, 8192, 16384, 16384, 11, hq=32, hkv=8, page=128, head_major=False,
            dtype="bf16"),
        # continuous batching: prompt chunks among decoding requests, three query heads to a key head
        _kv("mixed batch 64 requests", "attention", 64, 1, 2, 1, 6000, 12, hq=24, hkv=8, page=64, head_major=False,
            dtype="fp16", **{"chunks": 4, "chunk_hi": 512, "window": 2048, "sinks": 4}),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    seed = rng.randrange(1 << 20)
    op = rng.choice(["rope", "append", "read", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    head_major = rng.random() < 0.5
    if op == "rope":
        n_req = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, max(1, 32768 // n_req))
        hkv = rng.choice([1, 2, 4, 8])
        scaled = rng.random() < 0.5
        return {"op": op, "n_req": n_req, "new_lo": 0, "new_hi": hi, "old_lo": 0, "old_hi": _log_int(rng, 1, 1 << 20),
                "hq": hkv * rng.choice([1, 3, 4]), "hkv": hkv, "layout": rng.choice(["half", "pairs"]),
                "rot": rng.choice([128, 128, 96, 64, 32, 2 * rng.randint(1, 64)]), "base": rng.choice([1e4, 5e5, 1e6]),
                "factor": rng.uniform(1.5, 32.0) if scaled else 1.0, "original": rng.choice([0, 4096, 8192]) if scaled else 0,
                "dtype": dtype, "lens_seed": seed}
    if op in ("append", "read"):
        n_req = _log_int(rng, 1, 512)
        old = rng.choice([0, _log_int(rng, 1, 512)]) if op == "append" else 0
        most = 32768 if op == "append" else 65536
        new = _log_int(rng, 1, max(1, most // n_req))
        return {"op": op, "n_req": n_req, "new_lo": 1 if op == "read" else 0, "new_hi": new, "old_lo": 0, "old_hi": old,
                "chunks": 0, "chunk_hi": 1, "window": 0, "sinks": 0, "hkv": rng.choice([1, 2, 3, 5, 8]), "page": page,
                "head_major": head_major, "dtype": dtype, "lens_seed": seed}
    hkv = rng.choice([1, 2, 4, 8, 16])
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
        c["old_hi"] = rng.choice([0, _log_int(rng, 16, 16384)])
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
    if not sum(new):
        new[0] = 1
    return new, old


def _ceil(a, b):
    return -(-a // b)


# --- inputs ------------------------------------------------------------------

def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _exponent(amax):
    """Least e with amax <= 448 2^e (448 = 0.875 2^9), within the scales' range."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m > 0.875, e - 8, e - 9), LEAST).clamp(LEAST, MOST)


def _power(e):
    """2^e in 32 bits, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _eight(x):
    return x.clamp(-TOP, TOP).to(F8)


def _cache(case, n_pages, g, add=None):
    """8-bit k and v as [page, token, head, 128] views of token-major or head-major pages and their scales
    [page, head, block], filled with values whose size changes from block to block."""
    p, h = case["page"], case["hkv"]
    got = []
    for i in range(2):
        x = torch.empty((n_pages, h, p // BLOCK, BLOCK, D), dtype=torch.float16, device="cuda").normal_(generator=g)
        x *= torch.empty((n_pages, h, p // BLOCK, 1, 1), dtype=torch.float16, device="cuda").normal_(generator=g).mul_(0.5).exp_()
        if add is not None and i == 0:
            x[add[0].long(), :, 0, :4] += (0.5 * add[1])[None, :, None].half()
        amax = x.abs().amax((3, 4)).float()
        scale = _power(_exponent(amax))
        x = _eight(x.div_(scale[..., None, None].half())).view(n_pages, h, p, D)
        if not case["head_major"]:
            x = x.view(torch.uint8).permute(0, 2, 1, 3).contiguous().view(F8).permute(0, 2, 1, 3)
        got += [x.permute(0, 2, 1, 3), scale]
    return {"k_cache": got[0], "k_scale": got[1], "v_cache": got[2], "v_scale": got[3]}


def _pages(case, new, old, g):
    """Block table with the pages of each request in a random order, and how many there are."""
    owned = [_ceil(a + o, case["page"]) for a, o in zip(new, old)]
    n_pages = sum(owned) + 1
    order = torch.randperm(n_pages - 1, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + owned).cumsum(0)[:-1].cuda()
    col = torch.arange(max(owned), device="cuda")
    own_col = col[None] < torch.tensor(owned, device="cuda")[:, None]
    table = torch.where(own_col, order[(first[:, None] + col[None]).clamp(max=n_pages - 2)], -1)
    return table.to(torch.int32).contiguous(), n_pages


def _frequencies(case):
    """Radians a position of each pair, in 64 bits."""
    rot = case["rot"]
    f = case["base"] ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["original"]:  # pairs that turn often over the original context stay, slow ones are stretched
        w = ((case["original"] * f / (2 * math.pi) - 1.0) / 3.0).clamp(0, 1)
        return f * (w + (1 - w) / case["factor"])
    return f / case["factor"]


def _handles(s):
    """What a program keeps from its set-up on: the rotation's or the cache's handle, the workspace."""
    import linear_attention_serving_fwd_gb300 as kda

    c = s["case"]
    if c["op"] == "rope":
        f = kda.rope_frequencies(c["rot"], c["base"], factor=c["factor"], original_context=c["original"])
        s["rope"] = kda.Rope(f, layout=c["layout"])
        return
    s["cache"] = kda.KvCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], dtype=DTYPES[c["dtype"]])
    if c["op"] == "attention":
        s["workspace"] = kda.paged_attention_workspace("cuda", tokens=s["q"].shape[0], heads=c["hq"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    s = {"case": case}
    new, old = lens_of(case)
    t, dt = sum(new), DTYPES[case["dtype"]]
    kv = [a + o for a, o in zip(new, old)]
    s.update(cu_seqlens=torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda(), kv_lens=_int32(kv))
    if case["op"] == "rope":
        hq, hkv = case["hq"], case["hkv"]
        qkv = torch.empty((t, hq + 2 * hkv, D), dtype=dt, device="cuda").normal_(generator=g)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]  # bands of one projection
        s["frequencies"] = _frequencies(case).cuda()
    else:
        table, n_pages = _pages(case, new, old, g)
        hkv = case["hkv"]
        if case["op"] == "attention":
            # queries share a direction to which the prompt's first keys answer
            u = torch.empty((hkv, D), device="cuda").normal_(generator=g)
            q = torch.empty((t, case["hq"], D), device="cuda").normal_(generator=g)
            s["q"] = (q + u.repeat_interleave(case["hq"] // hkv, 0)).to(dt)
            s.update(_cache(case, n_pages, g, (table[[i for i, n in enumerate(kv) if n], 0], u)))
            s.update(table=table, scale=D ** -0.5)
        else:
            s.update(_cache(case, n_pages, g))
            of = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(new, device="cuda"))
            pos = torch.arange(t, device="cuda") - s["cu_seqlens"][of] + torch.tensor(old, device="cuda")[of]
            page = case["page"]
            s["slots"] = (table[of, pos // page] * page + pos % page).to(torch.int32)
            if case["op"] == "append":
                x = torch.empty((t, 2 * hkv, D), dtype=dt, device="cuda").normal_(generator=g)
                x *= torch.empty((t, 1, 1), dtype=dt, device="cuda").normal_(generator=g).exp_()
                s["k"], s["v"] = x[:, :hkv], x[:, hkv:]  # bands of one projection
    if own:
        _handles(s)
    torch.cuda.synchronize()
    return s


# --- one pass ----------------------------------------------------------------

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import linear_attention_serving_fwd_gb300 as kda

        if op == "rope":
            q, k = kda.kda_rope(s["rope"], s["q"], s["k"], cu_seqlens=s["cu_seqlens"], kv_lens=s["kv_lens"])
            return {"q": q, "k": k}
        if op == "append":
            kda.kda_kv_append(s["cache"], s["k"], s["v"], s["slots"])
            return {x: s[x] for x in ("k_cache", "k_scale", "v_cache", "v_scale")}
        if op == "read":
            k, v = kda.kda_kv_read(s["cache"], s["slots"])
            return {"k": k, "v": v}
        out, lse = kda.kda_paged_attention(s["cache"], s["q"], s["cu_seqlens"], s["kv_lens"], s["table"],
                                           scale=s["scale"], window=c["window"], sinks=c["sinks"], return_lse=True,
                                           workspace=s["workspace"])
        return {"out": out, "lse": lse}
    return {"rope": _rope_plain, "append": _append_plain, "read": _read_plain, "attention": _attention_plain}[op](s)


def _rope_plain(s):
    c, rot, cu = s["case"], s["case"]["rot"], s["cu_seqlens"]
    t = torch.arange(s["q"].shape[0], device=cu.device)
    of = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = s["kv_lens"][of] - (cu[of + 1] - t)
    # far positions: the angle in 64 bits
    angle = pos.double()[:, None] * s["frequencies"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        y = x.float()
        first = y[..., 0:rot:2] if c["layout"] == "pairs" else y[..., :rot // 2]
        second = y[..., 1:rot:2] if c["layout"] == "pairs" else y[..., rot // 2:rot]
        a, b = first * cos - second * sin, second * cos + first * sin
        both = torch.stack((a, b), -1).flatten(-2) if c["layout"] == "pairs" else torch.cat((a, b), -1)
        return torch.cat((both, y[..., rot:]), -1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _append_plain(s):
    c, slots = s["case"], s["slots"].long()
    p, h, per = c["page"], c["hkv"], c["page"] // BLOCK
    block, row = slots // BLOCK, slots % BLOCK
    n = s["k_scale"].shape[0] * per
    first = torch.full((n,), BLOCK, device=slots.device).scatter_reduce_(0, block, row, "amin")
    touched = block[row == first[block]]  # each once, by its first new token
    page, part, held = touched // per, touched % per, first[touched]
    earlier = torch.arange(BLOCK, device=slots.device)[None] < held[:, None]  # rows that hold tokens
    for name, x in (("k", s["k"]), ("v", s["v"])):
        cache, scale = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
        amax = torch.zeros((n, h), device=slots.device)
        amax.scatter_reduce_(0, block[:, None].expand(-1, h), x.float().abs().amax(-1), "amax")
        need = _power(_exponent(amax[touched]))
        was = scale[page, :, part]
        now = torch.where((held > 0)[:, None], torch.maximum(was, need), need)
        scale[page, :, part] = now
        blocks = cache.unflatten(1, (per, BLOCK))
        old = blocks[page, part]
        moved = _eight(old.view(F8).float() * (was / now)[:, None, :, None]).view(torch.uint8)
        blocks[page, part] = torch.where(earlier[:, :, None, None], moved, old)
        y = x.float() / scale[slots // p, :, slots % p // BLOCK][..., None]
        cache[slots // p, slots % p] = _eight(y).view(torch.uint8)
    return {x: s[x] for x in ("k_cache", "k_scale", "v_cache", "v_scale")}


def _read_plain(s):
    c, slots = s["case"], s["slots"].long()
    page, row = slots // c["page"], slots % c["page"]

    def values(name):
        x = s[name + "_cache"].view(torch.uint8)[page, row].view(F8).float() * s[name + "_scale"][page, :, row // BLOCK][..., None]
        return x.to(DTYPES[c["dtype"]])

    return {"k": values("k"), "v": values("v")}


def _attention_plain(s):
    c, q, cu, kv = s["case"], s["q"], s["cu_seqlens"], s["kv_lens"]
    new, _ = lens_of(c)
    b, hkv, t = c["n_req"], c["hkv"], q.shape[0]
    grp, most = c["hq"] // hkv, max(new)
    pages = s["table"].clamp(min=0)

    def values(name):  # [request, key head, key, 128] in 32 bits
        x = s[name + "_cache"].view(torch.uint8)[pages].view(F8).float().unflatten(2, (-1, BLOCK))
        x *= s[name + "_scale"][pages].transpose(2, 3)[:, :, :, None, :, None]
        return x.flatten(1, 3).transpose(1, 2)

    k, v = values("k"), values("v")
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
    new, old = lens_of(case)
    t, op, hkv = sum(new), case["op"], case["hkv"]
    if op == "rope":
        rows = t * (case["hq"] + hkv)
        return {"bytes": rows * D * 2 * 2 + 4 * (2 * len(new) + 1), "flops": rows * case["rot"] * 3}
    blocks = sum(_ceil(a + o, BLOCK) - o // BLOCK for a, o in zip(new, old) if a)
    if op == "append":
        return {"bytes": t * hkv * D * 2 * (2 + 1) + blocks * hkv * 2 * 4 + 4 * t, "flops": 0}
    if op == "read":
        return {"bytes": t * hkv * D * 2 * (2 + 1) + blocks * hkv * 2 * 4 + 4 * t, "flops": 0}
    w, sinks, hq = case["window"], case["sinks"], case["hq"]
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
    pages = sum(_ceil(a + o, case["page"]) for a, o in zip(new, old))
    return {"bytes": keys * hkv * 2 * D + keys * hkv * 2 * 4 // BLOCK + t * hq * (D * 2 * 2 + 4) + 4 * (2 * len(new) + pages),
            "flops": 4 * D * hq * pairs}


# --- the definition in 64 bits -----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope_exact, "append": _append_exact, "read": _read_exact, "attention": _attention_exact}[case["op"]](s)


def _rope_exact(s):
    c, rot = s["case"], s["case"]["rot"]
    new, old = lens_of(c)
    pos = torch.cat([torch.arange(o, o + a, dtype=torch.float64) for a, o in zip(new, old)]).cuda()
    turn = torch.polar(torch.ones_like(s["frequencies"]), s["frequencies"])  # one position's turn, for its angle
    angle = torch.outer(pos, turn.angle())
    spin = torch.complex(angle.cos(), angle.sin())[:, None]
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        pairs = torch.arange(rot, device=x.device).view(-1, 2) if c["layout"] == "pairs" else \
            torch.arange(rot, device=x.device).view(2, -1).T
        z = torch.complex(x[..., pairs[:, 0]], x[..., pairs[:, 1]]) * spin
        x[..., pairs[:, 0]], x[..., pairs[:, 1]] = z.real, z.imag
        got[name] = x
    return got


def _round_eight(x):
    """To the nearest number of 4 significant bits on a grid of 2^-9, ties to even, none past 448."""
    step = x.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52 << 52  # the power of two below
    step = step.view(torch.float64) / 8
    return ((x / step).round() * step).clamp(-TOP, TOP)


def _append_exact(s):
    c = s["case"]
    slots = s["slots"].tolist()
    powers = torch.tensor([2.0 ** e for e in range(LEAST, MOST + 1)], dtype=torch.float64, device="cuda")
    starts = [i for i, x in enumerate(slots) if i == 0 or x != slots[i - 1] + 1 or x % BLOCK == 0]
    got = {}
    for name in ("k", "v"):
        cache, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        for i, end in zip(starts, starts[1:] + [len(slots)]):
            page, at = divmod(slots[i], c["page"])
            block, row = divmod(at, BLOCK)
            x = s[name][i:end].double()  # the block's new tokens
            now = powers[torch.searchsorted(TOP * powers, x.abs().amax((0, 2)))]  # the least that reaches them
            if row:
                was = scale[page, :, block]
                now = torch.maximum(now, was)
                held = cache[page, at - row:at]
                cache[page, at - row:at] = torch.where((now > was)[None, :, None], _round_eight(held * (was / now)[:, None]), held)
            cache[page, at:at + end - i] = _round_eight(x / now[:, None])
            scale[page, :, block] = now
        got[name + "_cache"], got[name + "_scale"] = cache, scale
    return got


def _read_exact(s):
    c = s["case"]
    got = {}
    for name in ("k", "v"):
        x = s[name + "_cache"].permute(0, 2, 1, 3).double() * s[name + "_scale"].double().repeat_interleave(BLOCK, 2)[..., None]
        got[name] = x.permute(0, 2, 1, 3).flatten(0, 1)[s["slots"].long()]
    return got


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
            k, v = ((s[x + "_cache"].view(torch.uint8)[pages, :, h].view(F8).reshape(-1, D).double()
                     * s[x + "_scale"][pages, h].reshape(-1).double().repeat_interleave(BLOCK)[:, None])[:n] for x in "kv")
            for x in range(h * grp, (h + 1) * grp):
                w = (q[at:at + a, x].double() @ k.T) * s["scale"]
                w = torch.where(hidden, NEG, w)
                lse[at:at + a, x] = torch.logsumexp(w, -1)
                out[at:at + a, x] = torch.softmax(w, -1) @ v
        at += a
    return {"out": out, "lse": lse}
