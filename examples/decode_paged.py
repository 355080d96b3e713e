"""One attention layer that answers several requests at once from a paged cache.

    python examples/decode_paged.py

The prompts' keys and values are written in one call, then every step projects
the newest hidden states (tgemm_run), appends their keys and values, attends to
the whole cache, projects back, and, when a sequence outgrows its budget,
evicts the positions that have drawn the least attention into fresh pages.
Random weights; it prints what each part did.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_epilogue_02_gb300 as tg  # noqa: E402


class PagedLayer:
    """q_heads query heads over kv_heads key heads of `dim`; `pages` pages of
    page_size positions shared by `batch` sequences of at most `most` positions."""

    def __init__(self, batch, hidden, q_heads, kv_heads, dim, pages, page_size, most, e4m3=True, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.batch, self.q_heads, self.kv_heads, self.dim, self.dtype = batch, q_heads, kv_heads, dim, dtype
        out = (q_heads + 2 * kv_heads) * dim
        self.w_in = (torch.randn(hidden, out, device="cuda", generator=g) / hidden ** 0.5).to(dtype)
        self.w_out = (torch.randn(q_heads * dim, hidden, device="cuda", generator=g) / (q_heads * dim) ** 0.5).to(dtype)
        shape = (pages, page_size, kv_heads, dim)
        k, v = (torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn if e4m3 else dtype) for _ in range(2))
        scales = [torch.zeros(shape[:3], device="cuda") for _ in range(2)] if e4m3 else [None, None]
        self.cache = tg.PagedCache(k, v, *scales)
        self.free = list(range(pages))
        self.owned = [[] for _ in range(batch)]                  # each sequence's pages
        self.counts = [0] * batch                                # and positions, as the host knows them
        self.width = -(-most // page_size)
        self.weights = torch.zeros(batch, kv_heads, most, device="cuda")
        self.table = torch.zeros(batch, self.width, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.attended = torch.empty(batch, q_heads, dim, dtype=dtype, device="cuda")
        self.workspace = tg.attention_decode_workspace(self.attended, self.cache, self.table, weights=True)

    def _project(self, x):
        """Queries, keys and values of hidden states x [tokens, hidden], slices of one product."""
        out = torch.empty(x.shape[0], self.w_in.shape[1], dtype=self.dtype, device="cuda")
        tg.run(x, self.w_in, None, out, "none")
        out = out.view(x.shape[0], -1, self.dim)
        return out[:, :self.q_heads], out[:, self.q_heads:self.q_heads + self.kv_heads], out[:, self.q_heads + self.kv_heads:]

    def _grow(self, new):
        """Gives every sequence the pages for new[b] more positions."""
        for b, n in enumerate(new):
            self.counts[b] += n
            while len(self.owned[b]) * self.cache.page_size < self.counts[b]:
                self.owned[b].append(self.free.pop())
        self._publish()

    def _publish(self):
        rows = [p + [0] * (self.width - len(p)) for p in self.owned]
        self.table.copy_(torch.tensor(rows, dtype=torch.int32))
        self.lengths.copy_(torch.tensor(self.counts, dtype=torch.int32))

    def prompt(self, x, new):
        """Writes the keys and values of hidden states x [sum of new, hidden], new[b] of them sequence b's."""
        _, k, v = self._project(x)
        self._grow(new)
        starts = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        tg.kv_append(self.cache, k, v, self.table, self.lengths, starts=starts, weights=self.weights)

    def step(self, x):
        """The layer's output for one new hidden state per sequence, x [batch, hidden]."""
        q, k, v = self._project(x)
        self._grow([1] * self.batch)
        tg.kv_append(self.cache, k, v, self.table, self.lengths, weights=self.weights)
        tg.attention_decode(q, self.cache, self.table, self.lengths, self.attended, weights=self.weights,
                            workspace=self.workspace)
        out = torch.empty_like(x)
        tg.run(self.attended.view(self.batch, -1), self.w_out, None, out, "none")
        return out

    def trim(self, keep, recent):
        """Brings every sequence back to `keep` positions; returns the positions kept."""
        size = self.cache.page_size
        counts = [min(n, keep) for n in self.counts]
        fresh = [[self.free.pop() for _ in range(-(-n // size))] for n in counts]
        to_table = torch.tensor([p + [0] * (self.width - len(p)) for p in fresh], dtype=torch.int32, device="cuda")
        kept = torch.empty(self.batch, self.kv_heads, keep, dtype=torch.int32, device="cuda")
        to_weights = torch.zeros_like(self.weights)
        to_lengths = torch.empty_like(self.lengths)
        tg.kv_evict(self.cache, self.table, self.lengths, self.weights, self.cache, to_table, kept, to_lengths, to_weights,
                    recent=recent)
        for pages in self.owned:
            self.free.extend(pages)
        self.owned, self.counts, self.weights = fresh, counts, to_weights
        self._publish()
        return kept


def main(steps=40, budget=160):
    layer = PagedLayer(batch=4, hidden=512, q_heads=8, kv_heads=2, dim=64, pages=80, page_size=16, most=256)
    g = torch.Generator(device="cuda").manual_seed(1)
    new = [150, 1, 33, 97]
    layer.prompt(torch.randn(sum(new), 512, device="cuda", generator=g).to(layer.dtype), new)
    x = torch.randn(4, 512, device="cuda", generator=g).to(layer.dtype)
    for i in range(steps):
        x = layer.step(x)
        if max(layer.counts) > budget:
            layer.trim(keep=128, recent=32)
            print(f"step {i}: trimmed to {layer.counts}, {len(layer.free)} pages free")
    torch.cuda.synchronize()
    status = tg.tgemm_last_device_status()
    print(f"{steps} steps, positions {layer.counts}, output norm {x.float().norm().item():.3f}, device status {status}")
    return layer, status


if __name__ == "__main__":
    main()
