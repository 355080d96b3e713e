"""The paged cache's calls follow one another on a stream without a
synchronisation: each sees what all before it have written, eviction and the
added weights among them, again and again over the same memory."""
from __future__ import annotations

import pytest
import torch

import gemm_epilogue_02_gb300 as tg
from kv_helpers import E4M3

pytestmark = pytest.mark.gpu

HEADS, GROUP, DIM, PAGE, KEEP, ROOM = 4, 2, 64, 16, 96, 128


def chain(kind, wait, rounds=25):
    """Two pools in turn: each round appends to one, attends with weights, evicts into the other; small kernels of
    torch rewrite lengths and page lists between the rounds.  Every output of every round."""
    g = torch.Generator().manual_seed(17)
    ctype = E4M3 if kind == "e4m3" else torch.bfloat16
    width = ROOM // PAGE
    caches = []
    for _ in range(2):
        k, v = (torch.zeros(3 * width, PAGE, HEADS, DIM, device="cuda").to(ctype) for _ in range(2))
        sc = [torch.zeros(3 * width, PAGE, HEADS, device="cuda") for _ in range(2)] if kind == "e4m3" else [None, None]
        caches.append(tg.PagedCache(k, v, *sc))
    order = [torch.randperm(3 * width, generator=g).view(3, width).to(torch.int32).cuda()
             for _ in range(rounds + 1)]
    x = torch.randn(rounds, 3 * 40, HEADS, DIM, generator=g).bfloat16().cuda()
    q = torch.randn(rounds, 3, HEADS * GROUP, DIM, generator=g).bfloat16().cuda()
    table = order[0].clone()
    lengths = torch.zeros(3, dtype=torch.int32, device="cuda")
    weights = [torch.zeros(3, HEADS, ROOM, device="cuda") for _ in range(2)]
    starts = torch.tensor([0, 32, 47, 48], dtype=torch.int32, device="cuda")
    new = starts[1:] - starts[:-1]
    to_table, to_lengths = torch.empty_like(table), torch.empty_like(lengths)
    kept = torch.empty(3, HEADS, KEEP, dtype=torch.int32, device="cuda")
    o = torch.empty(3, HEADS * GROUP, DIM, dtype=torch.bfloat16, device="cuda")
    ws = tg.attention_decode_workspace(o, caches[0], table, weights=True)
    out = []

    def after():
        if wait:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    for i in range(rounds):
        a, b = caches[i % 2], caches[1 - i % 2]
        wa, wb = weights[i % 2], weights[1 - i % 2]
        lengths += new
        to_table.copy_(order[i + 1])
        after()
        tg.kv_append(a, x[i], x[i].flip(-1), table, lengths, starts=starts, weights=wa)
        after()
        for _ in range(2):
            tg.attention_decode(q[i], a, table, lengths, o, weights=wa, workspace=ws)
            after()
        tg.kv_evict(a, table, lengths, wa, b, to_table, kept, to_lengths, wb, recent=20)
        after()
        out += [o.clone(), wa.clone(), kept.clone(), to_lengths.clone(), wb[..., :KEEP].clone()]
        table.copy_(to_table)
        lengths.copy_(to_lengths)
        after()
    torch.cuda.synchronize()
    assert tg.tgemm_last_device_status() == 0
    assert lengths.tolist() == [min(KEEP, rounds * n) for n in new.tolist()]
    return out


@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_rounds_of_eviction_see_each_other(cuda_lib, kind):
    for a, b in zip(chain(kind, False), chain(kind, True)):
        assert torch.equal(a, b)
