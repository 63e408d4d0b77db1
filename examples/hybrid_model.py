"""A small hybrid model on one page table: recurrent layers on a paged state pool,
and every fourth layer attention on a paged key/value cache.

    python examples/hybrid_model.py [--prompts 700 130 1] [--chunk 256] [--tokens 8]

The prompts are fed in chunks (append with rotary positions, attention of the
chunk's tokens; the recurrent layers from the states their pages hold), then one
token per sequence is decoded at a time, greedily.  Weights and prompts are random.
The same prompts fed whole end in the same logits up to rounding, which the command prints.
"""

from __future__ import annotations

import argparse
import os
import sys
import time
from typing import List

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import paged_recurrent_state_amd as gdn  # noqa: E402

BF16 = torch.bfloat16


class Pages:
    """Page table of a batch whose sequences grow: page ids are given out in turn."""

    def __init__(self, seqs: int, page_size: int, device):
        self.page_size, self.device = page_size, device
        self.lengths, self.lists, self.used = [0] * seqs, [[] for _ in range(seqs)], 0

    def grow(self, new: List[int]):
        """The table after ``new`` more tokens of each sequence, and the tokens' cu_seqlens."""
        cu = [0]
        for b, n in enumerate(new):
            self.lengths[b] += n
            while len(self.lists[b]) * self.page_size < self.lengths[b]:
                self.lists[b].append(self.used)
                self.used += 1
            cu.append(cu[-1] + n)
        ptr = [0]
        for pages in self.lists:
            ptr.append(ptr[-1] + len(pages))
        last = [n - (len(p) - 1) * self.page_size if p else 0 for n, p in zip(self.lengths, self.lists)]
        i32 = dict(dtype=torch.int32, device=self.device)
        where = (torch.tensor(sum(self.lists, []), **i32), torch.tensor(ptr, **i32), self.page_size,
                 torch.tensor(last, **i32))
        return where, torch.tensor(cu, **i32)


class Model:
    def __init__(self, layers=4, hidden=512, heads=8, kv_heads=2, dim=128, rot=64, vocab=1024, pages=64,
                 page_size=128, window=0, softcap=0.0, positions=8192, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(n_in, n_out):
            return (torch.randn(n_in, n_out, generator=gen, device=device) * n_in ** -0.5).to(BF16)

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.attention = dict(window=window, softcap=softcap)
        self.table = gdn.rope_table(positions, rot, device=device)
        self.embedding = weight(vocab, hidden) * vocab ** 0.5
        self.head = weight(hidden, vocab)
        self.layers = []
        for i in range(layers):
            if i % 4 == 3:
                kv = torch.zeros(2, pages, page_size, kv_heads, dim, dtype=BF16, device=device)
                self.layers.append(dict(kind="attention", qkv=weight(hidden, (heads + 2 * kv_heads) * dim),
                                        out=weight(heads * dim, hidden), kv=kv))
            else:
                state = torch.zeros(pages, heads, dim, dim, device=device)
                self.layers.append(dict(kind="recurrent", qkv=weight(hidden, 3 * heads * dim),
                                        gates=weight(hidden, 2 * heads), out=weight(heads * dim, hidden), state=state))

    def _attend(self, w, x, where, cu):
        H, Hk = self.heads, self.kv_heads
        qkv = (x @ w["qkv"]).view(-1, H + 2 * Hk, self.dim)
        q, k, v = qkv.split([H, Hk, Hk], dim=1)  # views: the calls take their strides
        q = gdn.kv_append_paged(k, v, cu, *w["kv"], *where, table=self.table, q=q)
        if cu is None:
            return gdn.attention_decode_paged(q, *w["kv"], *where, **self.attention)
        return gdn.attention_prefill_paged(q, cu, *w["kv"], *where, **self.attention)

    def _recur(self, w, x, where, cu):
        q, k, v = (x @ w["qkv"]).view(-1, 3, self.heads, self.dim).unbind(1)
        q, k = (F.normalize(t.float(), dim=-1).to(BF16) for t in (q, k))
        a, b = (x @ w["gates"]).float().split(self.heads, dim=1)
        args = (q, k, v.contiguous(), -F.softplus(a - 3.0), torch.sigmoid(b))
        if cu is None:
            return gdn.decode_paged(*args, w["state"], *where)
        return gdn.prefill_paged(*args, cu, w["state"], *where)

    def step(self, tokens, where, cu=None):
        """Logits [T, vocab] of the batch's new tokens; ``cu`` None: one token per sequence."""
        x = self.embedding[tokens]
        for w in self.layers:
            y = F.rms_norm(x.float(), (x.shape[-1],)).to(BF16)
            o = (self._attend if w["kind"] == "attention" else self._recur)(w, y, where, cu)
            x = x + o.reshape(o.shape[0], -1) @ w["out"]
        return F.rms_norm(x.float(), (x.shape[-1],)).to(BF16) @ self.head

    def prompt(self, prompts, pages: Pages, chunk: int):
        """Feeds the prompts, ``chunk`` tokens of each at a time; logits of each one's last token."""
        last = [None] * len(prompts)
        for lo in range(0, max(len(t) for t in prompts), chunk):
            parts = [t[lo:lo + chunk] for t in prompts]
            where, cu = pages.grow([len(t) for t in parts])
            logits = self.step(torch.cat(parts), where, cu)
            at = 0
            for b, t in enumerate(parts):
                at += len(t)
                if len(t):
                    last[b] = logits[at - 1]
        return torch.stack(last)


def generate(prompts, chunk, tokens, seed=0, device="cuda", **kw):
    """(logits after the prompts, decoded tokens [B, tokens] (None: none asked for), logits after the last, the
    time of a decoded token)"""
    if not prompts or min(len(t) for t in prompts) < 1 or chunk < 1 or tokens < 0:
        raise ValueError("at least one prompt, of one token or more, chunks of one or more, and no fewer than 0 tokens")
    page_size = kw.setdefault("page_size", 128)
    need = sum(-(-(len(t) + tokens) // page_size) for t in prompts)
    model = Model(pages=need, device=device, seed=seed, positions=max(len(t) for t in prompts) + tokens, **kw)
    pages = Pages(len(prompts), page_size, device)
    first = logits = model.prompt(prompts, pages, chunk)
    out = []
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(tokens):
        out.append(logits.argmax(dim=-1))
        where, _ = pages.grow([1] * len(prompts))
        logits = model.step(out[-1], where)
    torch.cuda.synchronize()
    each = (time.perf_counter() - start) / max(1, tokens)
    return first, torch.stack(out, dim=1) if out else None, logits, each


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 130, 1])
    ap.add_argument("--chunk", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--softcap", type=float, default=0.0)
    a = ap.parse_args(argv)
    if min(a.prompts) < 1 or a.chunk < 1 or a.tokens < 0:
        ap.error("prompts and chunks have one token or more, and --tokens is 0 or more")
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1024, (n,), generator=gen).to("cuda") for n in a.prompts]
    kw = dict(window=a.window, softcap=a.softcap)
    first, out, _, each = generate(prompts, a.chunk, a.tokens, **kw)
    whole = generate(prompts, max(a.prompts), 0, **kw)[0]
    diff = ((first - whole).float().norm() / whole.float().norm()).item()
    print(f"{len(prompts)} prompts in chunks of {a.chunk}: logits within {diff:.1e} of the prompts fed whole")
    if out is not None:
        print(f"{a.tokens} tokens decoded, {1e3 * each:.2f} ms each")
        for t in out.tolist():
            print(" ", *t)


if __name__ == "__main__":
    main()
