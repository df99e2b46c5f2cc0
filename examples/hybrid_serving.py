"""Serving steps of a small hybrid model: recurrent KDA layers on a paged state
cache with a softmax-attention layer on a paged key/value cache after every
third of them.

    python examples/hybrid_serving.py

One request batch goes through prompt chunks of ragged lengths, decode steps,
a window of drafted tokens of which some are rejected, and release.  Weights
are random; the tokens are given, so that the same text can be run in steps of
other sizes and must give the same logits up to rounding.

Per step: kda_kv_extend takes pages for the step's tokens and lays them out;
in every layer the tokens are projected, and run through kda_chunk_fwd (prompt
chunks) or kda_decode (single tokens) on the request's state row, or written
with kda_kv_append and run through kda_paged_attention.  A rejected draft is
undone by kda_kv_truncate on the key/value side; on the recurrent side the
step is run from a copy of the states (kda_verify and kda_commit do that
without the copy).
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import linear_attention_serving_fwd_gb300 as kda

D = 128  # head dimension


class HybridModel:
    """Layers 0 .. n - 1; every fourth is softmax attention (``window`` > 0: of
    a sliding window with ``sinks`` first tokens that stay), the others KDA."""

    def __init__(self, n_layers=4, heads=8, kv_heads=2, vocab=512, window=0, sinks=0, requests=8, pages=64,
                 page_size=64, columns=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[0] ** -0.5).bfloat16()  # noqa: E731
        self.heads, self.kv_heads, self.hidden = heads, kv_heads, heads * D
        self.window, self.sinks = window, sinks
        self.embed, self.head = w(vocab, self.hidden) * vocab ** 0.5, w(self.hidden, vocab)
        self.layers = []
        for i in range(n_layers):
            if i % 4 == 3:
                kv = torch.zeros(2, pages, page_size, kv_heads, D, dtype=torch.bfloat16, device="cuda")
                self.layers.append(dict(kind="attention", qkv=w(self.hidden, (heads + 2 * kv_heads) * D),
                                        out=w(self.hidden, self.hidden), cache=kda.KvCache(kv[0], kv[1])))
            else:
                self.layers.append(dict(
                    kind="kda", proj=w(self.hidden, 4 * self.hidden + heads), out=w(self.hidden, self.hidden),
                    A_log=torch.zeros(heads, device="cuda"), dt_bias=torch.zeros(heads, D, device="cuda"),
                    states=torch.zeros(requests, heads, D, D, device="cuda")))
        self.pages = kda.KvPages.empty(requests, columns, pages, page_size)
        self.workspace = kda.paged_attention_workspace()
        self.rows = torch.arange(requests, dtype=torch.int32, device="cuda")

    def step(self, tokens, new_lens):
        """One step of the batch: ``tokens`` packed, new_lens[b] of request b
        (lists).  Returns the logits of all of them [T, vocab]."""
        lens = torch.tensor(new_lens, dtype=torch.int32, device="cuda")
        started = (self.pages.kv_lens > 0).to(torch.uint8)
        cu, slots, kv_lens = kda.kda_kv_extend(self.pages, lens, len(tokens))
        x = self.embed[torch.tensor(tokens, device="cuda")]
        for layer in self.layers:
            y = torch.nn.functional.rms_norm(x, (self.hidden,))
            y = self._attention(layer, y, cu, slots, kv_lens) if layer["kind"] == "attention" else \
                self._kda(layer, y, cu, started, max(new_lens))
            x = x + y.reshape(-1, self.hidden) @ layer["out"]
        return torch.nn.functional.rms_norm(x, (self.hidden,)) @ self.head

    def _attention(self, layer, y, cu, slots, kv_lens):
        qkv = (y @ layer["qkv"]).view(-1, self.heads + 2 * self.kv_heads, D)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        kda.kda_kv_append(layer["cache"], k, v, slots)
        return kda.kda_paged_attention(layer["cache"], q, cu, kv_lens, self.pages.block_table, window=self.window,
                                       sinks=self.sinks, workspace=self.workspace)[0]

    def _kda(self, layer, y, cu, started, longest):
        p = y @ layer["proj"]
        q, k, v, g = (p[:, i * self.hidden:(i + 1) * self.hidden].unflatten(1, (self.heads, D)) for i in range(4))
        beta = p[:, 4 * self.hidden:]
        gate = dict(A_log=layer["A_log"], dt_bias=layer["dt_bias"])
        if longest == 1:
            return kda.kda_decode(q, k, v, g, beta, layer["states"], cu, self.rows, 1, **gate)
        return kda.kda_chunk_fwd(q, k, v, g, beta, cu_seqlens=cu, state_cache=layer["states"],
                                 state_indices=self.rows, has_initial_state=started, **gate)[0]

    def states(self):
        return [layer["states"].clone() for layer in self.layers if layer["kind"] == "kda"]

    def restore(self, states):
        for layer, s in zip((x for x in self.layers if x["kind"] == "kda"), states):
            layer["states"].copy_(s)

    def rollback(self, keep_lens):
        kda.kda_kv_truncate(self.pages, torch.tensor(keep_lens, dtype=torch.int32, device="cuda"))


def serve(model, texts, chunk):
    """All texts through the model: prompts (all but the last eight tokens) in
    chunks, then a draft that is rejected, then token by token.  Returns each
    request's logits [len, vocab]."""
    n = len(texts)
    at, logits = [0] * n, [[] for _ in texts]

    def run(lens):
        out = model.step([t for b in range(n) for t in texts[b][at[b]:at[b] + lens[b]]], lens)
        for b, part in enumerate(out.split(lens)):
            logits[b].append(part)
            at[b] += lens[b]

    while any(at[b] < len(texts[b]) - 8 for b in range(n)):
        run([min(chunk, len(texts[b]) - 8 - at[b]) for b in range(n)])
    kept = model.states()
    model.step([7] * 4 * n, [4] * n)  # four drafted tokens, none of them accepted
    model.restore(kept)
    model.rollback(at)
    while any(at[b] < len(texts[b]) for b in range(n)):
        run([1] * n)
    model.rollback([0] * n)  # finished: all pages go back
    return [torch.cat(x) for x in logits]


def main():
    r = torch.Generator().manual_seed(3)
    texts = [torch.randint(512, (n,), generator=r).tolist() for n in (9, 40, 73, 137, 200, 300, 411, 650)]
    for window, sinks in ((0, 0), (96, 4)):
        whole, steps = (serve(HybridModel(window=window, sinks=sinks), texts, chunk) for chunk in (1000, 128))
        worst = max(float((a - b).float().norm() / a.float().norm()) for a, b in zip(whole, steps))
        model = HybridModel(window=window, sinks=sinks)
        serve(model, texts, 256)
        free = int(model.pages.free_count)
        status = kda.kda_device_status()
        print(f"window {window}, {sinks} sinks: prompts in chunks of 128 against whole prompts, logits differ by "
              f"{worst:.2e} (relative norm); {free} of 64 pages free at the end; device status {status}")
        assert worst < 5e-2 and free == 64 and status == 0


if __name__ == "__main__":
    main()
