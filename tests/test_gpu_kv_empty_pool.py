"""The paged cache's calls on a cache without pages: every position is left out
and reported, and a sequence of length 0 is answered with zeros."""
from __future__ import annotations

import pytest
import torch

from kv_helpers import E4M3

pytestmark = pytest.mark.gpu

CACHE = 9      # TGEMM_ERR_CACHE


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("width", [0, 3])
def test_a_cache_without_pages(cuda_lib, kind, width):
    tg = cuda_lib
    heads, dim, page = 2, 64, 16
    k, v = (torch.zeros(0, page, heads, dim, device="cuda").to(E4M3 if kind == "e4m3" else torch.bfloat16) for _ in range(2))
    sc = [torch.zeros(0, page, heads, device="cuda") for _ in range(2)] if kind == "e4m3" else [None, None]
    c = tg.PagedCache(k, v, *sc)
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    x = torch.ones(2, heads, dim, dtype=torch.bfloat16, device="cuda")
    lengths = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 2, 2], dtype=torch.int32, device="cuda")
    tg.kv_append(c, x, x, table, lengths + 1, starts=starts)
    assert tg.tgemm_last_device_status() == CACHE
    q = torch.ones(2, 4, dim, dtype=torch.bfloat16, device="cuda")
    for n, status in ((lengths, CACHE), (torch.zeros_like(lengths), 0)):
        o = torch.full_like(q, float("nan"))
        w = torch.full((2, heads, 48), 3.0, device="cuda")
        tg.attention_decode(q, c, table, n, o, weights=w)
        assert (o == 0).all() and (w == 3.0).all()
        assert tg.tgemm_last_device_status() == status
        kept = torch.empty(2, heads, 4, dtype=torch.int32, device="cuda")
        tl, tw = torch.empty_like(lengths), torch.empty(2, heads, 4, device="cuda")
        tg.kv_evict(c, table, n, w, c, table, kept, tl, tw)
        assert tg.tgemm_last_device_status() == status
