"""The paged cache's calls in graphs and on side streams: captured once and
replayed for the lengths, pages and weights found at each replay; on a stream
that other work of the same stream feeds."""
from __future__ import annotations

import pytest
import torch

import gemm_epilogue_02_gb300 as tg
from kv_helpers import E4M3

pytestmark = pytest.mark.gpu

HEADS, DIM, PAGE, BATCH = 3, 64, 16, 3


def new_cache(kind, pages):
    t = E4M3 if kind == "e4m3" else torch.bfloat16
    k, v = (torch.zeros(pages, PAGE, HEADS, DIM, device="cuda").to(t) for _ in range(2))
    sc = [torch.zeros(pages, PAGE, HEADS, device="cuda") for _ in range(2)] if kind == "e4m3" else [None, None]
    return tg.PagedCache(k, v, *sc)


def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def everything(c):
    return [t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("tokens", [1, 40])
def test_appending_in_a_graph(cuda_lib, kind, tokens):
    g = torch.Generator().manual_seed(1)
    pages = BATCH * 8
    table = torch.randperm(pages, generator=g).to(torch.int32).view(BATCH, 8).cuda()
    K, V = (torch.empty(BATCH * tokens, HEADS, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lengths = torch.full((BATCH,), tokens, dtype=torch.int32, device="cuda")
    starts = None if tokens == 1 else torch.zeros(BATCH + 1, dtype=torch.int32, device="cuda")
    captured, plain = new_cache(kind, pages), new_cache(kind, pages)
    w = [torch.ones(BATCH, HEADS, 8 * PAGE, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tg.kv_append(captured, K, V, table, lengths, starts=starts, weights=w[0])
    for i in range(4):
        for t in (K, V):
            t.copy_(torch.randn(t.shape, generator=g))
        table.copy_(table[:, torch.randperm(8, generator=g).cuda()])
        if starts is not None:
            counts = torch.tensor([[40, 40, 40], [1, 100, 19], [0, 0, 120], [3, 0, 7]][i])
            starts[1:] = counts.cumsum(0).to(torch.int32).cuda()
            lengths.copy_(counts + i)
        else:
            lengths.copy_(torch.tensor([[1, 1, 1], [17, 2, 128], [64, 65, 3], [9, 9, 9]][i]))
        graph.replay()
        tg.kv_append(plain, K, V, table, lengths, starts=starts, weights=w[1])
        torch.cuda.synchronize()
        assert all(same_bytes(a, b) for a, b in zip(everything(captured), everything(plain)))
        assert torch.equal(*w) and (w[0] == 0).any()
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("kind,width,most", [("16", 32, 500), ("e4m3", 32, 500), ("16", 700, 11000), ("e4m3", 4200, 60000)])
def test_eviction_in_a_graph(cuda_lib, kind, width, most):
    """Selections by one block and by clusters of two and of eight."""
    g = torch.Generator().manual_seed(2)
    keep = 90
    source = new_cache(kind, BATCH * width)
    for t in everything(source):
        if t.dtype == E4M3:
            t.view(torch.uint8).copy_(torch.randint(0, 127, t.shape, generator=g, dtype=torch.uint8))
        else:
            t.copy_(torch.randn(t.shape, generator=g))
    table = torch.randperm(BATCH * width, generator=g).to(torch.int32).view(BATCH, width).cuda()
    lengths = torch.zeros(BATCH, dtype=torch.int32, device="cuda")
    weights = torch.zeros(BATCH, HEADS, width * PAGE, device="cuda")
    to_table = torch.arange(BATCH * 6, dtype=torch.int32).view(BATCH, 6).cuda()
    outs = []
    for _ in range(2):
        outs.append((new_cache(kind, BATCH * 6), torch.zeros(BATCH, HEADS, keep, dtype=torch.int32, device="cuda"),
                     torch.zeros(BATCH, dtype=torch.int32, device="cuda"), torch.zeros(BATCH, HEADS, keep, device="cuda")))

    def call(to, kept, to_lengths, to_weights):
        tg.kv_evict(source, table, lengths, weights, to, to_table, kept, to_lengths, to_weights, recent=11)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*outs[0])
    for i, n in enumerate(([most, 3, 91], [0, most // 2, 90], [200, 201, most])):
        lengths.copy_(torch.tensor(n))
        weights.copy_((torch.rand(weights.shape, generator=g) * 50).floor())
        graph.replay()
        call(*outs[1])
        torch.cuda.synchronize()
        for a, b in zip(outs[0][1:], outs[1][1:]):
            assert torch.equal(a, b)
        assert outs[0][2].tolist() == [min(x, keep) for x in n]
        assert all(same_bytes(a, b) for a, b in zip(everything(outs[0][0]), everything(outs[1][0])))
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_all_calls_on_a_side_stream(cuda_lib, kind):
    """Inputs made on the side stream just before, outputs read on it just after, by its current stream and by the
    argument; a long kernel in front keeps the stream busy, so that work on another stream would come too early."""
    results = []
    for how in ("default", "current", "argument"):
        g = torch.Generator().manual_seed(3)
        c, to = new_cache(kind, BATCH * 8), new_cache(kind, BATCH * 4)
        table = torch.arange(BATCH * 8, dtype=torch.int32).view(BATCH, 8).cuda()
        to_table = torch.arange(BATCH * 4, dtype=torch.int32).view(BATCH, 4).cuda()
        x = torch.randn(2, BATCH * 30, HEADS, DIM, generator=g).bfloat16().cuda()
        K, V = torch.zeros_like(x[0]), torch.zeros_like(x[1])
        q0 = torch.randn(BATCH, 2 * HEADS, DIM, generator=g).bfloat16().cuda()
        q, o = torch.zeros_like(q0), torch.zeros_like(q0)
        starts = torch.zeros(BATCH + 1, dtype=torch.int32, device="cuda")
        lengths = torch.zeros(BATCH, dtype=torch.int32, device="cuda")
        w = torch.full((BATCH, HEADS, 8 * PAGE), 9.0, device="cuda")
        kept = torch.zeros(BATCH, HEADS, 20, dtype=torch.int32, device="cuda")
        tl, tw = torch.zeros_like(lengths), torch.zeros(BATCH, HEADS, 20, device="cuda")
        begin = torch.tensor([0, 30, 60, 90], dtype=torch.int32, device="cuda")
        big = torch.ones(4096, 4096, device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        stream = None if how == "default" else side
        with torch.cuda.stream(stream if how != "default" else torch.cuda.current_stream()):
            for _ in range(3):
                big = big @ big * 1e-4
            starts.copy_(begin)
            lengths += begin[1]
            K.copy_(x[0])
            V.copy_(x[1])
            q.copy_(q0)
            if how != "argument":
                tg.kv_append(c, K, V, table, lengths, starts=starts, weights=w)
                tg.attention_decode(q, c, table, lengths, o, weights=w)
                tg.kv_evict(c, table, lengths, w, to, to_table, kept, tl, tw, recent=4)
        if how == "argument":
            tg.kv_append(c, K, V, table, lengths, starts=starts, weights=w, stream=side)
            tg.attention_decode(q, c, table, lengths, o, weights=w, stream=side)
            tg.kv_evict(c, table, lengths, w, to, to_table, kept, tl, tw, recent=4, stream=side)
        with torch.cuda.stream(stream if how != "default" else torch.cuda.current_stream()):
            results.append([t.clone() for t in (o, w, kept, tl, tw, *everything(c), *everything(to))])
        torch.cuda.synchronize()
    assert (results[0][3] == 20).all() and torch.isfinite(results[0][0].float()).all() and (results[0][0] != 0).any()
    for other in results[1:]:
        assert all(same_bytes(a, b) for a, b in zip(results[0], other))
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("lengths", [[900, 64, 5], [9000, 300, 1], [100] * 40])
def test_a_sequence_does_not_depend_on_what_its_neighbours_hold(cuda_lib, kind, lengths):
    """The same first sequence beside neighbours of the same lengths and other contents: the same bits; and alone:
    the same but for the order of its sums."""
    g = torch.Generator().manual_seed(4)
    width = -(-max(lengths) // PAGE)
    table = torch.arange(len(lengths) * width, dtype=torch.int32).view(len(lengths), width).cuda()
    first = torch.randn(2, lengths[0], HEADS, DIM, generator=g).bfloat16().cuda()
    q = torch.randn(len(lengths), 4 * HEADS, DIM, generator=g).bfloat16().cuda()
    outs = []
    for case in ("one", "other", "alone"):
        ns = lengths[:1] if case == "alone" else lengths
        c = new_cache(kind, len(ns) * width)
        rows = [torch.cat([first[i]] + [torch.randn(n, HEADS, DIM, generator=g).bfloat16().cuda() * (5 if case == "other" else 1)
                                        for n in ns[1:]]) for i in range(2)]
        starts = torch.tensor([sum(ns[:b]) for b in range(len(ns) + 1)], dtype=torch.int32, device="cuda")
        n = torch.tensor(ns, dtype=torch.int32, device="cuda")
        tg.kv_append(c, rows[0], rows[1], table[:len(ns)], n, starts=starts)
        qq = q[:len(ns)].clone()
        if case == "other":
            qq[1:] *= -2
        o = torch.empty_like(qq)
        tg.attention_decode(qq, c, table[:len(ns)], n, o)
        outs.append(o[0].float().cpu())
    assert torch.equal(outs[0], outs[1])
    # Alone, the sums are ordered otherwise: a few roundings of fp32 and of each weight's parts, then one of bf16.
    assert ((outs[0] - outs[2]).abs() <= 2.0 ** -7 * outs[0].abs() + 2.0 ** -12).all()
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 256])
def test_appending_rows_that_are_not_finite(cuda_lib, dim, dtype):
    """e4m3: a NaN stays one and does not count in its row's scale; an infinity makes the scale infinite, its row's
    finite elements 0 and itself NaN; other rows are as without them."""
    g = torch.Generator().manual_seed(5)
    n, heads = 64, 2
    x = torch.randn(n, heads, dim, generator=g).to(dtype)
    nan, inf, all_nan = slice(0, 8), slice(8, 16), slice(16, 18)
    for j in range(8):
        x[j, 0, (5 * j) % dim] = float("nan")
        x[8 + j, 1, (7 * j) % dim] = float("inf") if j % 2 else float("-inf")
    x[all_nan] = float("nan")
    k, v = (torch.zeros(4, PAGE, heads, dim, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.zeros(4, PAGE, heads, device="cuda") for _ in range(2))
    tg.kv_append(tg.PagedCache(k, v, ks, vs), x.cuda(), x.flip(0).cuda(), torch.arange(4, dtype=torch.int32).view(1, 4).cuda(),
                 torch.tensor([n], dtype=torch.int32).cuda(), starts=torch.tensor([0, n], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for pool, scale, rows in ((k, ks, x), (v, vs, x.flip(0))):
        rows = rows.float()
        isnan = torch.isnan(rows)
        top = torch.where(isnan, torch.zeros_like(rows), rows).abs().amax(-1)
        want = torch.where(top > 0, top / 448.0, torch.ones_like(top))
        got_s, got = scale.view(n, heads).cpu(), pool.view(n, heads, dim).float().cpu()
        assert torch.equal(got_s, want)
        quotient = rows / want.unsqueeze(-1)
        assert torch.equal(torch.isnan(got), torch.isnan(quotient))
        fine = ~torch.isnan(quotient)
        assert torch.equal(got[fine], quotient.to(E4M3).float()[fine])
    assert tg.tgemm_last_device_status() == 0
