"""One attention layer that draws several continuations of each prompt from a paged cache and reads only the pages that matter.

    python examples/decode_samples.py

Pages are handed out, shared, freed and moved on the device: a prompt is written once and its continuations are forks of
it, which share its full pages. Every step grows the sequences by a token, normalises and rotates the newest queries and keys
by position, appends, bounds the keys of pages that are full, selects pages by them and attends to those. Random weights; it
prints what each part did.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_epilogue_02_gb300 as tg  # noqa: E402


class SamplingLayer:
    """q_heads query heads over kv_heads key heads of `dim`; `rows` sequences, prompts and their continuations, of at most
    `most` positions on `pages` pages; attention reads at most `keep` pages of each."""

    def __init__(self, rows, hidden, q_heads, kv_heads, dim, pages, page_size, most, keep, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim, self.dtype = q_heads, kv_heads, dim, dtype
        out = (q_heads + 2 * kv_heads) * dim
        self.w_in = (torch.randn(hidden, out, device="cuda", generator=g) / hidden ** 0.5).to(dtype)
        self.w_out = (torch.randn(q_heads * dim, hidden, device="cuda", generator=g) / (q_heads * dim) ** 0.5).to(dtype)
        self.q_norm, self.k_norm = (torch.ones(dim, dtype=dtype, device="cuda") for _ in range(2))
        self.rotary = tg.Rotary([10000.0 ** (-2 * i / dim) for i in range(dim // 2)])
        k, v = (torch.zeros(pages, page_size, kv_heads, dim, dtype=dtype, device="cuda") for _ in range(2))
        self.cache = tg.PagedCache(k, v)
        self.bounds = tg.PageBounds(torch.zeros(pages, kv_heads, 2, dim, dtype=torch.int8, device="cuda"),
                                    torch.ones(pages, kv_heads, device="cuda"))
        self.uses = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.table = torch.zeros(rows, -(-most // page_size), dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.chosen = torch.zeros(rows, kv_heads, keep, dtype=torch.int32, device="cuda")
        self.chosen_lengths = torch.zeros_like(self.lengths)
        self.attended = torch.empty(rows, q_heads, dim, dtype=dtype, device="cuda")
        self.workspace = tg.attention_decode_workspace(self.attended, self.cache, self.chosen)

    def _write(self, x, rows, positions, shift, starts=None, tokens=None):
        """Grows the sequences `rows`, and writes the keys and values of hidden states x [tokens, hidden] to their ends;
        returns the queries."""
        table, lengths = self.table[rows], self.lengths[rows]
        tg.kv_grow(self.cache, self.uses, table, lengths, tokens=tokens)
        out = torch.empty(x.shape[0], self.w_in.shape[1], dtype=self.dtype, device="cuda")
        tg.run(x, self.w_in, None, out, "none")
        out = out.view(x.shape[0], -1, self.dim)
        q, k, v = out[:, :self.q_heads], out[:, self.q_heads:self.q_heads + self.kv_heads], out[:, self.q_heads + self.kv_heads:]
        tg.qk_norm_rope(q, k, lengths if positions is None else positions, self.rotary, q, k, q_weight=self.q_norm,
                        k_weight=self.k_norm, shift=shift)
        tg.kv_append(self.cache, k, v, table, lengths, starts=starts)
        tg.kv_bounds(self.cache, self.bounds, table, lengths, starts=starts)
        return q

    def prompt(self, x, new):
        """Writes hidden states x [sum of new, hidden] as the first new[b] positions of sequences 0 .. len(new) - 1."""
        counts = torch.tensor(new, dtype=torch.int32, device="cuda")
        starts = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        positions = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in new])
        self._write(x, slice(0, len(new)), positions, 0, starts, counts)

    def branch(self, parents, first):
        """Sequences first, first + 1, ... give back what they hold and continue sequences `parents`."""
        rows = slice(first, first + len(parents))
        tg.kv_free(self.cache, self.uses, self.table[rows], self.lengths[rows])
        tg.kv_fork(self.cache, self.uses, self.table, self.lengths, torch.tensor(parents, dtype=torch.int32, device="cuda"),
                   self.table[rows], self.lengths[rows])

    def step(self, x):
        """The layer's output for one new hidden state of each sequence, x [rows, hidden]."""
        q = self._write(x, slice(None), None, -1)              # the newest position is the length that counts it, less one
        tg.kv_select(q, self.cache, self.bounds, self.table, self.lengths, self.chosen, self.chosen_lengths, first=1, recent=2)
        tg.attention_decode(q, self.cache, self.chosen, self.chosen_lengths, self.attended, workspace=self.workspace)
        out = torch.empty_like(x)
        tg.run(self.attended.view(x.shape[0], -1), self.w_out, None, out, "none")
        return out

    def compact(self):
        """Moves the pages in use to the front of the pool; returns how many they are."""
        in_use = torch.empty(1, dtype=torch.int32, device="cuda")
        tg.kv_compact(self.cache, self.uses, self.table, self.lengths, self.table, self.uses, in_use, bounds=self.bounds)
        return int(in_use)


def main(steps=30):
    layer = SamplingLayer(rows=8, hidden=512, q_heads=8, kv_heads=2, dim=64, pages=160, page_size=16, most=512, keep=8)
    g = torch.Generator(device="cuda").manual_seed(1)
    new = [300, 77]
    layer.prompt(torch.randn(sum(new), 512, device="cuda", generator=g).to(layer.dtype), new)
    layer.branch([0, 0, 0, 1, 1, 1], first=2)
    x = torch.randn(8, 512, device="cuda", generator=g).to(layer.dtype)
    for _ in range(steps):
        x = layer.step(x)
    layer.branch([3, 3], first=4)                              # two samples end, another goes on twice
    for _ in range(steps):
        x = layer.step(x)
    used = layer.compact()
    x = layer.step(x)
    torch.cuda.synchronize()
    status = tg.tgemm_last_device_status()
    print(f"positions {layer.lengths.tolist()} on {used} pages, output norm {x.float().norm().item():.3f}, device status {status}")
    return layer, used, status


if __name__ == "__main__":
    main()
