"""The paged cache's operators together, as they would be used: the example's
layer step by step against the definitions, the debug build's checks, and calls
back to back with other work on the stream."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import gemm_epilogue_02_gb300 as tg
from gemm_epilogue_02_gb300 import kv
from kv_helpers import E4M3, Filled, attend64, attend_bound, make_pool, make_table

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def rows_of(layer, b):
    """Sequence b's keys and values in 64 bits, read from the cache: [n, heads, dim] each."""
    n, size, c = layer.counts[b], layer.cache.page_size, layer.cache
    pos = torch.arange(n, device="cuda")
    page, slot = layer.table[b].long()[pos // size], pos % size
    out = []
    for pool, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        if scale is None:
            out.append(pool[page, slot].double().cpu())
        else:
            out.append((pool.view(torch.uint8)[page, slot].view(E4M3).double() * scale[page, slot].double().unsqueeze(-1)).cpu())
    return out


@pytest.mark.parametrize("e4m3", [True, False])
def test_layer_of_the_example_step_by_step(cuda_lib, e4m3):
    """Every step's attention is that of the rows in the cache; the newest rows are the projected ones; eviction
    keeps the rows that it says, and their weights."""
    from decode_paged import PagedLayer
    layer = PagedLayer(batch=3, hidden=256, q_heads=6, kv_heads=2, dim=64, pages=60, page_size=8, most=120, e4m3=e4m3)
    g = torch.Generator(device="cuda").manual_seed(3)
    new = [70, 0, 9]
    layer.prompt(torch.randn(sum(new), 256, device="cuda", generator=g).to(layer.dtype), new)
    seen = []
    real = layer._project

    def spy(x):
        seen[:] = [t.double().cpu() for t in real(x)]
        return real(x)
    layer._project = spy
    x = torch.randn(3, 256, device="cuda", generator=g).to(layer.dtype)
    for i in range(12):
        x = layer.step(x)
        torch.cuda.synchronize()
        for b in range(3):
            k, v = rows_of(layer, b)
            step = 2.0 ** -4 if e4m3 else 0.0
            assert ((k[-1] - seen[1][b]).abs() <= step * seen[1][b].abs() + seen[1][b].abs().amax() * 2.0 ** -17).all()
            o, p, mag, reach, top = attend64(seen[0][b], k, v, 64 ** -0.5)
            bound = attend_bound(o, mag, reach, top, len(k), 64, "bf16", "fp16" if e4m3 else "bf16", 0.0)
            assert ((layer.attended[b].double().cpu() - o).abs() <= bound).all(), (i, b)
        if i == 6:
            before = [rows_of(layer, b) for b in range(3)]
            weights = layer.weights.clone()
            kept = layer.trim(keep=40, recent=10)
            torch.cuda.synchronize()
            for b in range(3):
                after = rows_of(layer, b)
                for h in range(2):
                    idx = kept[b, h, :layer.counts[b]].long().cpu()
                    for a, c in zip(after, before[b]):
                        assert torch.equal(a[:, h], c[idx, h])
                    assert torch.equal(layer.weights[b, h, :layer.counts[b]].cpu(), weights[b, h].cpu()[idx])
    assert sum(len(p) for p in layer.owned) + len(layer.free) == 60
    assert cuda_lib.tgemm_last_device_status() == 0


def test_example_runs(cuda_lib):
    from decode_paged import main
    layer, status = main(steps=25, budget=160)
    assert status == 0 and max(layer.counts) <= 160


def both_libraries(monkeypatch, call):
    """call() through the release and the debug library: both results, and the debug one's status and check id."""
    results = []
    for lib in (tg.load(), tg.load_debug()):
        for name in ("tgemm_kv_append", "tgemm_attention_decode", "tgemm_kv_evict"):
            f = getattr(lib, name)

            def through(args, stream=0, f=f):
                return f(args, stream)
            through.__name__ = name
            monkeypatch.setattr(kv._b, name, through)
        results.append(call())
        torch.cuda.synchronize()
    dbg = tg.load_debug()
    assert dbg.tgemm_last_device_status() == 0 and dbg.tgemm_debug_last_check() == 0
    return results


@pytest.mark.parametrize("cache,dtype,dim,group", [("16", "fp16", 64, 1), ("16", "bf16", 128, 12), ("e4m3", "bf16", 80, 8),
                                                   ("e4m3", "fp16", 256, 3)])
def test_debug_build_finds_nothing_and_agrees(cuda_lib, monkeypatch, cache, dtype, dim, group):
    def call():
        f = Filled(cuda_lib, [700, 0, 3, 5000], 2, dim, 16, dtype, cache, seed=dim)
        g = torch.Generator().manual_seed(5)
        q = torch.randn(4, 2 * group, dim, generator=g).to(torch.float16 if dtype == "fp16" else torch.bfloat16).cuda()
        o, w = torch.empty_like(q), torch.rand(4, 2, 5000, generator=g).cuda()
        tg.attention_decode(q, f.cache, f.table, f.lengths, o, weights=w,
                            workspace=tg.attention_decode_workspace(q, f.cache, f.table, weights=True))
        to_table, pages = make_table([min(n, 100) for n in f.lengths_host], 16, 0, 9)
        k, v = make_pool(pages, 16, 2, dim, f.k.dtype, "pshd", "cuda")
        sc = [torch.zeros(pages, 16, 2, device="cuda") for _ in range(2)] if cache == "e4m3" else [None, None]
        kept = torch.empty(4, 2, 100, dtype=torch.int32, device="cuda")
        tl, tw = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(4, 2, 100, device="cuda")
        to = tg.PagedCache(k, v, *sc)
        tg.kv_evict(f.cache, f.table, f.lengths, w, to, to_table.cuda(), kept, tl, tw, recent=20)
        x = torch.randn(4, 2, dim, generator=g).to(q.dtype).cuda()
        lengths = torch.tensor([100, 1, 3, 50], dtype=torch.int32).cuda()
        to_table[1, 0] = to_table[0, 0]      # a fresh sequence on a page that the first no longer needs
        tg.kv_append(to, x, x, to_table.cuda(), lengths, weights=tw)
        return [t.clone() for t in (o, w, kept, tl, tw)] + [t.view(torch.uint8).clone() for t in (k, v)]
    a, b = both_libraries(monkeypatch, call)
    for s, t in zip(a, b):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_calls_back_to_back_see_each_other(cuda_lib):
    """Append, attention and eviction chained without a synchronisation, against the same with one after each call
    (kernels may begin before the previous one has ended; none may read before it has)."""
    def chain(wait):
        f = Filled(tg, [900, 40, 1], 4, 128, 16, "bf16", "e4m3", seed=31, width=64, extra=40)
        g = torch.Generator().manual_seed(6)
        free = [p for p in range(f.k.shape[0]) if p not in set(f.table_host.flatten().tolist())]
        for b, n in enumerate(f.lengths_host):      # room for the new tokens
            have = -(-n // 16)
            f.table[b, have:have + 4] = torch.tensor(free[4 * b:4 * b + 4], dtype=torch.int32)
        q = torch.randn(3, 16, 128, generator=g).bfloat16().cuda()
        w = torch.rand(3, 4, 1024, generator=g).cuda()
        o = [torch.empty_like(q) for _ in range(20)]
        ws = tg.attention_decode_workspace(q, f.cache, f.table, weights=True)
        kept = torch.empty(3, 4, 64, dtype=torch.int32, device="cuda")
        tl, tw = torch.empty(3, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, 64, device="cuda")
        k, v = make_pool(12, 16, 4, 128, E4M3, "pshd", "cuda")
        sc = [torch.zeros(12, 16, 4, device="cuda") for _ in range(2)]
        to = tg.PagedCache(k, v, *sc)
        to_table = torch.arange(12, dtype=torch.int32).view(3, 4).cuda()
        torch.cuda.synchronize()
        for i in range(20):
            f.lengths += 1
            kvs = q[:, :4] * (1 + 0.1 * i)
            tg.kv_append(f.cache, kvs, kvs, f.table, f.lengths, weights=w)
            if wait:
                torch.cuda.synchronize()
            tg.attention_decode(q, f.cache, f.table, f.lengths, o[i], weights=w, workspace=ws)
            if wait:
                torch.cuda.synchronize()
        tg.kv_evict(f.cache, f.table, f.lengths, w, to, to_table, kept, tl, tw, recent=9)
        if wait:
            torch.cuda.synchronize()
        tg.attention_decode(q, to, to_table, tl, o[0], workspace=ws)
        torch.cuda.synchronize()
        assert tg.tgemm_last_device_status() == 0
        return o + [w, kept, tl, tw]
    for a, b in zip(chain(False), chain(True)):
        assert torch.equal(a, b)


def test_a_scale_of_zero_stands_for_values_of_zero(cuda_lib):
    f = Filled(cuda_lib, [50, 7], 2, 64, 16, "bf16", "e4m3", seed=41)
    for b, j in ((0, 3), (0, 20), (1, 0)):
        page = int(f.table_host[b, j // 16])
        f.ks[page, j % 16] = 0
        f.vs[page, j % 16] = 0
        f.k64[b][j], f.v64[b][j] = 0, 0
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(7)).bfloat16()
    out = torch.empty_like(q, device="cuda")
    tg.attention_decode(q.cuda(), f.cache, f.table, f.lengths, out)
    for b, n in enumerate((50, 7)):
        o, p, mag, reach, top = attend64(q[b], f.k64[b], f.v64[b], 0.125)
        bound = attend_bound(o, mag, reach, top, n, 64, "bf16", "fp16", 0.0)
        assert ((out[b].double().cpu() - o).abs() <= bound).all()


def test_scales_far_apart(cuda_lib):
    """Value scales over forty powers of two: each weight keeps its relative precision, and the largest rows theirs."""
    f = Filled(cuda_lib, [300], 1, 64, 16, "bf16", "e4m3", seed=42)
    g = torch.Generator().manual_seed(8)
    for j in range(300):
        page, factor = int(f.table_host[0, j // 16]), 2.0 ** int(torch.randint(-30, 10, (1,), generator=g))
        f.vs[page, j % 16] *= factor
        f.v64[0][j] *= factor
    q = torch.randn(1, 4, 64, generator=g).bfloat16()
    out, w = torch.empty_like(q, device="cuda"), torch.zeros(1, 1, 300, device="cuda")
    tg.attention_decode(q.cuda(), f.cache, f.table, f.lengths, out, weights=w)
    o, p, mag, reach, top = attend64(q[0], f.k64[0], f.v64[0], 0.125)
    bound = attend_bound(o, mag, reach, top, 300, 64, "bf16", "fp16", 0.0)
    assert ((out[0].double().cpu() - o).abs() <= bound).all()
    assert ((w[0, 0].double().cpu() - p.sum(0)).abs() <= 2e-5 * p.sum(0)).all()
