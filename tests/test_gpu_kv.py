"""GPU parity of the paged key-value cache's operators with their definitions
in 64 bits (kv_helpers): appending, attention of one new token, eviction.
Unused rows of every cache hold NaN and unused page numbers lie outside the
pool, so that reading either shows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_helpers import (E4M3, TDT, Filled, attend64, attend_bound, evict_reference, make_pool, make_table,
                        score_error, split_e4m3)

pytestmark = pytest.mark.gpu

CACHE = 9      # TGEMM_ERR_CACHE


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


# ---------------------------------------------------------------- append
def run_append(tg, context, new, heads, dim, page, dtype, cache, layout, with_starts=True, pad=0, stride_heads=0, seed=0):
    """Appends to a poisoned cache and compares every byte of both pools and of the scales and weights."""
    lengths = [c + n for c, n in zip(context, new)]
    table, pages = make_table(lengths, page, 2, seed)
    ctype = E4M3 if cache == "e4m3" else TDT[dtype]
    k, v = make_pool(pages, page, heads, dim, ctype, layout, "cuda")
    ks = vs = None
    if cache == "e4m3":
        ks, vs = (torch.full((pages, page, heads), float("nan"), device="cuda") for _ in range(2))
    T, B = sum(new) + 2 * pad, len(new)
    g = torch.Generator().manual_seed(seed)
    # Keys and values as slices of one projection's output [tokens, heads + stride_heads, 2 * dim].
    x = torch.randn(T, heads + stride_heads, 2, dim, generator=g)
    x[::3] *= 100
    x[1::5, 0] = 0
    x = x.to(TDT[dtype])
    xd = x.cuda()
    K, V = xd[:, :heads, 0], xd[:, :heads, 1]
    starts = torch.tensor([pad + sum(new[:b]) for b in range(B + 1)], dtype=torch.int32)
    weights = torch.full((B, heads, max(1, max(lengths))), 5.0, device="cuda")
    want_w = weights.cpu().clone()
    want = [bits(t).clone() for t in (k, v) + ((ks, vs) if ks is not None else ())]
    tok = pad
    for b in range(B):
        for i in range(new[b]):
            pos = context[b] + i
            pg, slot = int(table[b, pos // page]), pos % page
            for w, src in enumerate((x[tok, :heads, 0], x[tok, :heads, 1])):
                if cache == "e4m3":
                    e, s = split_e4m3(src)
                    want[w][pg, slot] = e.view(torch.uint8)
                    want[2 + w][pg, slot] = s.view(torch.int32)
                else:
                    want[w][pg, slot] = src.contiguous().view(torch.int16)
            want_w[b, :, pos] = 0
            tok += 1
    tg.kv_append(tg.PagedCache(k, v, ks, vs), K, V, table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                 starts=starts.cuda() if with_starts else None, weights=weights)
    torch.cuda.synchronize()
    for got, w in zip((k, v) + ((ks, vs) if ks is not None else ()), want):
        assert torch.equal(bits(got), w)
    assert torch.equal(weights.cpu(), want_w)
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("cache,dtype", [("16", "fp16"), ("16", "bf16"), ("e4m3", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("layout", ["pshd", "phsd", "both"])
@pytest.mark.parametrize("dim,heads,page", [(64, 8, 16), (128, 2, 7), (80, 3, 1), (256, 1, 24)])
def test_append_ragged(cuda_lib, dim, heads, page, layout, cache, dtype):
    run_append(cuda_lib, [0, 5, 31, 2, 0], [3, 0, 1, 40, 1], heads, dim, page, dtype, cache, layout, pad=2,
               stride_heads=1, seed=dim + page)


@pytest.mark.parametrize("cache", ["16", "e4m3"])
@pytest.mark.parametrize("batch", [1, 2, 33, 300])
def test_append_one_token_each(cuda_lib, batch, cache):
    run_append(cuda_lib, [(7 * b) % 50 for b in range(batch)], [1] * batch, 4, 64, 16, "bf16", cache, "pshd",
               with_starts=False, seed=batch)


def test_append_many_tokens(cuda_lib):
    run_append(cuda_lib, [3, 0, 1], [1500, 1, 700], 2, 128, 32, "fp16", "e4m3", "phsd", seed=4)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_e4m3_quotients_of_every_magnitude(cuda_lib, dtype):
    """Rows whose largest element runs over the type's whole range, subnormals among them, with elements from it
    down: scales and elements are those of the definition, bit for bit."""
    tg = cuda_lib
    heads, dim, page, n = 4, 256, 16, 700
    g = torch.Generator().manual_seed(21)
    lo, hi = (-24, 15) if dtype == "fp16" else (-133, 127)
    top = torch.exp2(lo + (hi - lo) * torch.rand(n, heads, 1, generator=g, dtype=torch.float64))
    x = top * torch.exp2(-12 * torch.rand(n, heads, dim, generator=g, dtype=torch.float64))
    x *= torch.randint(0, 2, x.shape, generator=g) * 2 - 1
    x[:, :, 7] = top[:, :, 0]
    x = x.to(TDT[dtype])
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    k, v = make_pool(n // page + 1, page, heads, dim, E4M3, "pshd", "cuda")
    ks, vs = (torch.full((n // page + 1, page, heads), float("nan"), device="cuda") for _ in range(2))
    table = torch.arange(n // page + 1, dtype=torch.int32).view(1, -1).cuda()
    tg.kv_append(tg.PagedCache(k, v, ks, vs), x.cuda(), -x.flip(0).cuda(), table,
                 torch.tensor([n], dtype=torch.int32).cuda(), starts=torch.tensor([0, n], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for pool, scale, rows in ((k, ks, x), (v, vs, -x.flip(0))):
        e, s = split_e4m3(rows)
        assert torch.equal(scale.view(-1, heads)[:n].cpu().view(torch.int32), s.view(torch.int32))
        assert torch.equal(pool.view(torch.uint8).view(-1, heads, dim)[:n].cpu(), e.view(torch.uint8))
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_append_bad_pages_and_lengths_are_left_out(cuda_lib, cache):
    """A page outside the pool, a length that does not reach back to position 0, and one past the page list: their
    tokens are left out and reported, the others are written."""
    tg = cuda_lib
    heads, dim, page = 2, 64, 4
    k, v = make_pool(6, page, heads, dim, E4M3 if cache == "e4m3" else torch.float16, "pshd", "cuda")
    sc = [torch.full((6, page, heads), float("nan"), device="cuda") for _ in range(2)] if cache == "e4m3" else [None, None]
    table = torch.tensor([[0, 6], [1, -1], [2, 3], [4, 5]], dtype=torch.int32)
    # tokens per sequence 2, 2, 3, 2; lengths: 6 (page 6 is outside), 5 (page -1 holds position 4), 2 (token 0 before 0), 9 (past 8)
    starts = torch.tensor([0, 2, 4, 7, 9], dtype=torch.int32)
    lengths = torch.tensor([6, 5, 2, 9], dtype=torch.int32)
    x = torch.ones(9, heads, dim, dtype=torch.float16, device="cuda")
    tg.kv_append(tg.PagedCache(k, v, *sc), x, x, table.cuda(), lengths.cuda(), starts=starts.cuda())
    torch.cuda.synchronize()
    assert tg.tgemm_last_device_status() == CACHE
    written = (~torch.isnan(k.float())).all(-1).all(-1).nonzero().tolist()
    assert written == [[1, 3], [2, 0], [2, 1], [5, 3]]


# ---------------------------------------------------------------- attend
def run_attend(tg, f, q_heads, cap=0.0, window=0, with_weights=False, scale=None, q_gain=1.0, seed=1, keep=None, stream=None,
               workspace="own", q_strided=False):
    """Runs attention_decode on a Filled cache and compares with the definition."""
    B, dim = len(f.lengths_host), f.dim
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, q_heads, dim, generator=g) * q_gain).to(TDT[f.dtype])
    if q_strided:   # a slice of a wider projection, and an output with padded rows
        qd = torch.full((B, q_heads + 3, dim), float("nan"), dtype=TDT[f.dtype], device="cuda")[:, :q_heads]
        qd.copy_(q)
        out = torch.full((q_heads, B, dim + 8), float("nan"), dtype=TDT[f.dtype], device="cuda").transpose(0, 1)[..., :dim]
    else:
        qd, out = q.cuda(), torch.full((B, q_heads, dim), float("nan"), dtype=TDT[f.dtype], device="cuda")
    scale = dim ** -0.5 if scale is None else scale
    most = max([1] + f.lengths_host)
    w = torch.rand(B, f.heads, most + 3, generator=g) if with_weights else None
    wd = w.cuda() if with_weights else None
    ws = tg.attention_decode_workspace(qd, f.cache, f.table, weights=with_weights) if workspace == "own" else workspace
    torch.cuda.synchronize()
    tg.attention_decode(qd, f.cache, f.table, f.lengths, out, scale=scale, cap=cap, window=window, weights=wd,
                        workspace=ws, stream=stream)
    torch.cuda.synchronize()
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    p_dtype = "fp16" if f.kind == "e4m3" else f.dtype
    for b, n in enumerate(f.lengths_host):
        lo = max(0, n - window) if window else 0
        idx = torch.arange(lo, n) if keep is None else torch.tensor([j for j in keep[b] if j >= lo], dtype=torch.long)
        o, p, mag, reach, top = attend64(q[b], f.k64[b][:n], f.v64[b][:n], scale, cap, idx)
        bound = attend_bound(o, mag, reach, top, n, dim, f.dtype, p_dtype, cap)
        bad = (got[b] - o).abs() > bound
        assert not bad.any(), (b, n, int(bad.sum()), float(((got[b] - o).abs() - bound).max()))
        if idx.numel() == 0:
            assert (got[b] == 0).all()
        if with_weights:
            add = p.view(f.heads, q_heads // f.heads, n).sum(1)
            e = (2 * score_error(reach, dim, cap) + 2 * (n + 64) * 2.0 ** -24).view(f.heads, -1).amax(-1, keepdim=True)
            want = w[b].double()
            want[:, :n] += add
            allowed = 2.0 ** -22 * want
            allowed[:, :n] += 2 * e * add
            diff = (wd[b].double().cpu() - want).abs()
            assert (diff <= allowed).all(), (b, n, float((diff - allowed).max()))
            untouched = torch.ones(most + 3, dtype=torch.bool)
            untouched[idx] = False
            assert torch.equal(wd[b].cpu()[:, untouched], w[b][:, untouched])
    return out, wd


KINDS = [("16", "fp16"), ("16", "bf16"), ("e4m3", "fp16"), ("e4m3", "bf16")]


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 12, 17])
def test_attend_dims_and_groups(cuda_lib, dim, group, cache, dtype):
    f = Filled(cuda_lib, [1, 77, 300], 2, dim, 16, dtype, cache, seed=dim + group)
    run_attend(cuda_lib, f, 2 * group, with_weights=group in (3, 12))
    assert cuda_lib.tgemm_last_device_status() == 0


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("page", [1, 2, 5, 8, 16, 20, 64, 1024])
def test_attend_pages(cuda_lib, page, cache, dtype):
    f = Filled(cuda_lib, [130, 15, 16, 17, 128], 3, 64, page, dtype, cache, seed=page)
    run_attend(cuda_lib, f, 6, with_weights=True)
    assert cuda_lib.tgemm_last_device_status() == 0


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("layout", ["phsd", "both"])
def test_attend_layouts_and_strides(cuda_lib, layout, cache, dtype):
    f = Filled(cuda_lib, [200, 1, 63], 4, 128, 16, dtype, cache, layout=layout, seed=3)
    run_attend(cuda_lib, f, 8, q_strided=True)


@pytest.mark.parametrize("lengths", [[0], [0, 0, 5], [1], [2], [0, 1, 0, 1000, 0], [15, 16, 17, 31, 32, 33, 127, 128, 129],
                                     [4097, 1, 2500]])
def test_attend_lengths(cuda_lib, lengths):
    f = Filled(cuda_lib, lengths, 2, 64, 16, "fp16", seed=len(lengths))
    run_attend(cuda_lib, f, 4, with_weights=True)
    assert cuda_lib.tgemm_last_device_status() == 0


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("window", [1, 7, 16, 100, 5000])
def test_attend_window(cuda_lib, window, cache, dtype):
    f = Filled(cuda_lib, [0, 3, 200, 1111], 2, 64, 8, dtype, cache, seed=window)
    run_attend(cuda_lib, f, 8, window=window, with_weights=True)


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("cap", [0.5, 30.0])
def test_attend_capped(cuda_lib, cap, cache, dtype):
    f = Filled(cuda_lib, [40, 700], 2, 128, 16, dtype, cache, seed=5, k_gain=3.0)
    run_attend(cuda_lib, f, 8, cap=cap, with_weights=True, q_gain=3.0)


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("cap", [200.0, 1e4, 1e6, 1e12, 1e19, 1e30, 1e300])
def test_attend_large_caps(cuda_lib, cap, cache, dtype):
    """A cap far above the scores leaves them as they are: the error of a capped
    score goes by the score, not by the cap.  tanh's relative error, in units of
    2^-24: the series 5 roundings; 1 - 2 / (1 + 2^x) from x = -1/2 or 1/2 on
    (tanh >= 0.17) 2 for 2^x, 5 q + 1 for the rest with q <= 1.17: at most 48 of tanh."""
    dim, n = 128, 700
    f = Filled(cuda_lib, [n], 2, dim, 16, dtype, cache, seed=5, k_gain=3.0)
    q = (torch.randn(1, 8, dim, generator=torch.Generator().manual_seed(2)) * 3.0).to(TDT[dtype])
    out, w = torch.empty_like(q, device="cuda"), torch.zeros(1, 2, n, device="cuda")
    cuda_lib.attention_decode(q.cuda(), f.cache, f.table, f.lengths, out, cap=cap, weights=w)
    o, p, mag, reach, top = attend64(q[0], f.k64[0], f.v64[0], dim ** -0.5, cap)
    like = 3 * reach.clamp(max=cap)          # 48 units of the score as 16 of a cap
    bound = attend_bound(o, mag, reach, top, n, dim, dtype, "fp16" if cache == "e4m3" else dtype, like)
    assert ((out[0].double().cpu() - o).abs() <= bound).all()
    add = p.view(2, 4, n).sum(1)
    e = (2 * score_error(reach, dim, like) + 2 * (n + 64) * 2.0 ** -24).view(2, 4).amax(-1, keepdim=True)
    assert ((w[0].double().cpu() - add).abs() <= (2.0 ** -22 + 2 * e) * add).all()


@pytest.mark.parametrize("cap", [1e-30, 1e-45, 1e-300])
def test_attend_caps_near_zero(cuda_lib, cap):
    """Scores that all become 0: the average of the values, with keys that give a score of 0 among them."""
    f = Filled(cuda_lib, [100], 1, 64, 16, "bf16", seed=8)
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    q[0, 1] = 0
    out = torch.empty_like(q, device="cuda")
    cuda_lib.attention_decode(q.cuda(), f.cache, f.table, f.lengths, out, cap=cap)
    o, p, mag, reach, top = attend64(q[0], f.k64[0], f.v64[0], 0.0)
    assert ((out[0].double().cpu() - o).abs() <= attend_bound(o, mag, reach, top, 100, 64, "bf16", "bf16", 0.0)).all()


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_attend_peaked_and_other_scales(cuda_lib, scale, cache, dtype):
    """scale 1 makes scores of a few tens: the softmax is close to one-hot and
    the running maximum moves; a negative one turns the order round."""
    f = Filled(cuda_lib, [500, 2100], 2, 64, 16, dtype, cache, seed=6, k_gain=2.0)
    run_attend(cuda_lib, f, 4, scale=scale, q_gain=2.0)


@pytest.mark.parametrize("cache,dtype", KINDS)
def test_attend_long_tail(cuda_lib, cache, dtype):
    """One position outweighs each other one by about 2^26, and the answer is theirs alone: rounded to fp16 a weight
    may be off by 2^-25 of what is 1, and the largest weight is at least 2^7.  Rows that one block each takes."""
    n, dim, batch, heads = 600, 64, 8, 38
    f = Filled(cuda_lib, [n] * batch, heads, dim, 16, dtype, cache, seed=9)
    pages = f.table_host[:, 0].long().cuda()
    if cache == "e4m3":
        f.k.view(torch.uint8)[pages, 0] = 0x7E     # 448
        f.ks[pages, 0] = 8.0 / 448.0
        f.v.view(torch.uint8).fill_(0x38)          # 1
        f.v.view(torch.uint8)[pages, 0] = 0
        f.vs.fill_(1.0)
    else:
        f.k[pages, 0] = 8.0
        f.v.fill_(1.0)
        f.v[pages, 0] = 0.0
    q, scale = torch.ones(batch, heads, dim, dtype=TDT[dtype]), 26 * 0.6931 / 512
    out = torch.empty_like(q, device="cuda")
    cuda_lib.attention_decode(q.cuda(), f.cache, f.table, f.lengths, out, scale=scale)
    for b in range(batch):
        f.k64[b][0], f.v64[b][:] = 8.0, 1.0
        f.v64[b][0] = 0.0
        o, p, mag, reach, top = attend64(q[b], f.k64[b], f.v64[b], scale)
        bound = attend_bound(o, mag, reach, top * 2.0 ** -7, n, dim, dtype, "fp16" if cache == "e4m3" else dtype, 0.0)
        assert ((out[b].double().cpu() - o).abs() <= bound).all()


def test_attend_one_sequence_split_over_the_gpu(cuda_lib):
    """One key head: the whole GPU works on one row, joined in two levels."""
    f = Filled(cuda_lib, [50000], 1, 64, 16, "bf16", seed=7)
    run_attend(cuda_lib, f, 3, with_weights=True)


@pytest.mark.parametrize("lengths", [[700, 0, 33], [3000], [50] * 40 + [900]])
@pytest.mark.parametrize("cache,dtype,group", [("16", "fp16", 1), ("e4m3", "bf16", 3), ("16", "bf16", 12)])
def test_attend_more_heads_than_share_a_run(cuda_lib, lengths, cache, dtype, group):
    """So many key heads that every block goes through several of them."""
    f = Filled(cuda_lib, lengths, 72, 32, 16, dtype, cache, seed=len(lengths))
    run_attend(cuda_lib, f, 72 * group, with_weights=group == 3)
    assert cuda_lib.tgemm_last_device_status() == 0


def test_attend_many_heads_on_one(cuda_lib):
    """Blocks of heads beyond three eights, and three eights at once where the work is long."""
    for group, n in ((33, 300), (48, 5000), (24, 40000), (71, 90)):
        f = Filled(cuda_lib, [n, 7], 1, 64, 16, "bf16", seed=group)
        run_attend(cuda_lib, f, group, with_weights=True)


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 80, 96, 128])
@pytest.mark.parametrize("group,width", [(9, 2000), (12, 4000), (16, 2000), (17, 2000), (24, 2000), (24, 4000), (33, 4000), (39, 4000)])
def test_attend_several_eights_of_heads(cuda_lib, group, width, dim, cache, dtype):
    """Page lists that could hold long contexts: a block takes two or three eights of heads."""
    f = Filled(cuda_lib, [1, 77, 1500], 2, dim, 16, dtype, cache, seed=dim + group, width=width)
    run_attend(cuda_lib, f, 2 * group, with_weights=group in (9, 24), cap=30.0 if group == 16 else 0.0)
    assert cuda_lib.tgemm_last_device_status() == 0


def test_attend_large_batch(cuda_lib):
    lengths = [(37 * b) % 150 for b in range(700)]
    f = Filled(cuda_lib, lengths, 2, 64, 16, "bf16", seed=8)
    run_attend(cuda_lib, f, 4)


def test_attend_is_deterministic_and_leaves_its_workspace_fit(cuda_lib):
    tg = cuda_lib
    a = Filled(tg, [3000, 10, 777], 2, 128, 16, "bf16", seed=9)
    b = Filled(tg, [1, 2, 1500], 2, 128, 16, "bf16", seed=10)
    q = torch.randn(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = tg.attention_decode_workspace(q, a.cache, a.table)
    outs = []
    for f in (a, b, a, a, b):
        o = torch.empty_like(q)
        tg.attention_decode(q, f.cache, f.table, f.lengths, o, workspace=ws)
        outs.append(bits(o))
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[0], outs[3]) and torch.equal(outs[1], outs[4])


def test_attend_does_not_depend_on_neighbours(cuda_lib):
    """A sequence alone and in a batch: the same within twice the bound (the split differs)."""
    f = Filled(cuda_lib, [900, 64, 5], 2, 64, 16, "fp16", seed=11)
    run_attend(cuda_lib, f, 4)
    g = Filled(cuda_lib, [900], 2, 64, 16, "fp16", seed=11)
    assert torch.equal(f.k64[0], g.k64[0])
    run_attend(cuda_lib, g, 4)


@pytest.mark.parametrize("cache,dtype", KINDS)
def test_attend_bad_pages_are_left_out(cuda_lib, cache, dtype):
    """Pages outside the pool count as missing positions: the rest of the row answers, and the status tells."""
    tg = cuda_lib
    f = Filled(tg, [100, 40, 16], 2, 64, 16, dtype, cache, seed=12)
    f.table[0, 2] = -1
    f.table[0, 6] = f.k.shape[0]
    f.table[2, 0] = 0x7FFFFFFF
    keep = [[j for j in range(100) if j // 16 not in (2, 6)], list(range(40)), []]
    run_attend(tg, f, 4, with_weights=True, keep=keep)
    assert tg.tgemm_last_device_status() == CACHE
    assert tg.tgemm_last_device_status() == 0


def test_attend_bad_lengths(cuda_lib):
    """A negative length counts as 0; one past the page list as what the list can hold."""
    tg = cuda_lib
    f = Filled(tg, [32, 64, 10], 1, 64, 16, "fp16", seed=13, width=4)
    f.lengths.copy_(torch.tensor([-5, 1000, 10], dtype=torch.int32))
    f.lengths_host = [0, 64, 10]
    run_attend(tg, f, 2, with_weights=True)
    assert tg.tgemm_last_device_status() == CACHE


def test_attend_weights_narrower_than_a_sequence(cuda_lib):
    """Positions past the weights' width are left out of them and reported; the output is whole."""
    tg = cuda_lib
    f = Filled(tg, [50], 1, 64, 16, "fp16", seed=14)
    q = torch.randn(1, 2, 64, dtype=torch.float16, device="cuda")
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    w = torch.zeros(1, 1, 64, device="cuda")
    wide = torch.zeros(1, 1, 64, device="cuda")
    tg.attention_decode(q, f.cache, f.table, f.lengths, o, weights=w[:, :, :40])
    assert tg.tgemm_last_device_status() == CACHE
    tg.attention_decode(q, f.cache, f.table, f.lengths, o2, weights=wide)
    assert tg.tgemm_last_device_status() == 0
    assert torch.equal(o, o2) and torch.equal(w[..., :40], wide[..., :40]) and (w[..., 40:] == 0).all()


def test_attend_infinite_and_nan_rows_outside_the_window(cuda_lib):
    f = Filled(cuda_lib, [64], 1, 64, 16, "fp16", seed=15)
    for j in range(40):
        pg = int(f.table_host[0, j // 16])
        f.k[pg, j % 16] = float("inf") if j % 2 else float("nan")
        f.v[pg, j % 16] = float("nan") if j % 2 else float("-inf")
    run_attend(cuda_lib, f, 4, window=24)


def test_attend_nan_of_a_used_row_shows(cuda_lib):
    """A NaN in a row that counts reaches the outputs of its own head and no other."""
    f = Filled(cuda_lib, [64, 64], 2, 64, 16, "fp16", seed=16)
    f.v[int(f.table_host[0, 1]), 3, 1, 5] = float("nan")
    q = torch.randn(2, 4, 64, dtype=torch.float16, device="cuda")
    o = torch.zeros_like(q)
    cuda_lib.attention_decode(q, f.cache, f.table, f.lengths, o)
    nan = torch.isnan(o).cpu()
    assert nan[0, 2:, 5].all() and int(nan.sum()) == 2


def test_attend_on_another_stream_and_in_a_graph(cuda_lib):
    """Captured once, replayed for other lengths; without a workspace and with one; on a side stream."""
    tg = cuda_lib
    f = Filled(tg, [500, 33], 2, 64, 16, "bf16", seed=17)
    side = torch.cuda.Stream()
    run_attend(tg, f, 4, stream=side, workspace=None)
    q = torch.randn(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, want = torch.zeros_like(q), torch.zeros_like(q)
    w = torch.zeros(2, 2, 500, device="cuda")
    ws = tg.attention_decode_workspace(q, f.cache, f.table, weights=True)
    lengths = f.lengths.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tg.attention_decode(q, f.cache, f.table, lengths, o, weights=w, workspace=ws)
    for case in ([500, 33], [1, 0], [64, 20]):
        lengths.copy_(torch.tensor(case, dtype=torch.int32))
        w.zero_()
        o.fill_(float("nan"))
        graph.replay()
        wanted = torch.zeros_like(w)
        tg.attention_decode(q, f.cache, f.table, lengths, want, weights=wanted)
        torch.cuda.synchronize()
        assert torch.equal(bits(o), bits(want)) and torch.equal(w, wanted)


# ---------------------------------------------------------------- evict
def run_evict(tg, lengths, heads, dim, page, dtype, cache, keep, recent, weights=None, to_page=None, layout="pshd", seed=0,
              same_pool=False):
    f = Filled(tg, lengths, heads, dim, page, dtype, cache, layout=layout, seed=seed,
               extra=2 + (sum(-(-min(n, keep) // page) for n in lengths) if same_pool else 0))
    B = len(lengths)
    g = torch.Generator().manual_seed(seed + 1)
    most = max([1] + lengths)
    if weights is None:
        weights = (torch.rand(B, heads, most, generator=g) ** 4 * 8).mul(16).floor().div(16)     # many ties
    w = torch.full((B, heads, most + 2), float("inf"))
    w[:, :, :most] = weights
    want_k = [min(n, keep) for n in lengths]
    to_page = page if to_page is None else to_page
    if same_pool:
        used = set(f.table_host[f.table_host != 0x7FFFFFFF].tolist())
        free = [p for p in range(f.k.shape[0]) if p not in used]
        to_table, _ = make_table(want_k, page, 0, seed + 2)
        to_table = torch.tensor([[free[p] if p != 0x7FFFFFFF else p for p in row] for row in to_table.tolist()],
                                dtype=torch.int32)
        to, tk, tv, tks, tvs = f.cache, f.k, f.v, f.ks, f.vs
    else:
        to_table, to_pages = make_table(want_k, to_page, 1, seed + 2)
        tk, tv = make_pool(to_pages, to_page, heads, dim, f.k.dtype, "phsd" if layout == "pshd" else "pshd", "cuda")
        tks = tvs = None
        if cache == "e4m3":
            tks, tvs = (torch.full((to_pages, to_page, heads), float("nan"), device="cuda") for _ in range(2))
        to = tg.PagedCache(tk, tv, tks, tvs)
    before = [bits(t).clone() for t in (f.k, f.v)]
    kept = torch.full((B, heads, keep), -7, dtype=torch.int32, device="cuda")
    to_lengths = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    to_w = torch.full((B, heads, keep + 1), 99.0, device="cuda")
    tg.kv_evict(f.cache, f.table, f.lengths, w.cuda(), to, to_table.cuda(), kept, to_lengths, to_w, recent=recent)
    torch.cuda.synchronize()
    assert to_lengths.tolist() == want_k
    assert (to_w[..., keep] == 99.0).all()
    pools = [(bits(a), bits(b)) for a, b in ((f.k, tk), (f.v, tv))]
    scales = [(f.ks.cpu(), tks.cpu()), (f.vs.cpu(), tvs.cpu())] if cache == "e4m3" else []
    for b, n in enumerate(lengths):
        k = want_k[b]
        for h in range(heads):
            ref = evict_reference(w[b, h].numpy(), n, keep, recent)
            assert kept[b, h, :k].tolist() == ref and (kept[b, h, k:] == -1).all(), (b, h)
            got_w, want_w = to_w[b, h, :keep].cpu(), torch.zeros(keep)
            want_w[:k] = w[b, h, ref]
            assert torch.equal(got_w.view(torch.int32), want_w.view(torch.int32))
            src, dst = torch.tensor(ref, dtype=torch.long), torch.arange(k)
            sp, ss = f.table_host[b].long()[src // page], src % page
            dp, ds = to_table[b].long()[dst // to_page], dst % to_page
            for a, c in pools:
                assert torch.equal(c[dp, ds, h], a[sp, ss, h])
            for a, c in scales:
                assert torch.equal(c[dp, ds, h], a[sp, ss, h])
    if not same_pool:
        for t, old in zip((f.k, f.v), before):
            assert torch.equal(bits(t), old)
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (64, 0), (64, 16), (64, 64), (64, 100), (200, 31)])
def test_evict(cuda_lib, keep, recent, cache, dtype):
    run_evict(cuda_lib, [300, 0, 64, 65, 1, 63], 2, 64, 16, dtype, cache, keep, recent, to_page=8, seed=keep + recent)


@pytest.mark.parametrize("cache", ["16", "e4m3"])
@pytest.mark.parametrize("dim,page,layout", [(80, 5, "pshd"), (128, 1, "phsd"), (256, 32, "both")])
def test_evict_layouts(cuda_lib, dim, page, layout, cache):
    run_evict(cuda_lib, [150, 90], 3, dim, page, "bf16", cache, 77, 10, layout=layout, seed=dim)


def test_evict_within_one_pool(cuda_lib):
    run_evict(cuda_lib, [130, 70], 2, 64, 16, "fp16", "16", 48, 8, same_pool=True, seed=3)


@pytest.mark.parametrize("n,keep", [(5000, 1024), (3001, 3000), (9001, 1), (40000, 2048), (70001, 7)])
def test_evict_long(cuda_lib, n, keep):
    run_evict(cuda_lib, [n], 1, 64, 16, "fp16", "16", keep, min(keep // 2, 100), seed=n)


def test_evict_with_room_for_very_long_sequences(cuda_lib):
    """A page list and weights that could hold more keys than the selection keeps in shared memory: they are read
    again in each pass."""
    tg = cuda_lib
    n, keep, room = 9000, 700, 400016
    f = Filled(tg, [n, 650], 2, 64, 16, "fp16", seed=22, width=room // 16)
    w = torch.rand(2, 2, room, generator=torch.Generator().manual_seed(23)).mul(64).floor()
    to_table, pages = make_table([keep, 650], 16, 0, 3)
    tk, tv = make_pool(pages, 16, 2, 64, torch.float16, "pshd", "cuda")
    kept = torch.empty(2, 2, keep, dtype=torch.int32, device="cuda")
    tl, tw = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, 2, keep, device="cuda")
    tg.kv_evict(f.cache, f.table, f.lengths, w.cuda(), tg.PagedCache(tk, tv), to_table.cuda(), kept, tl, tw, recent=50)
    torch.cuda.synchronize()
    assert tl.tolist() == [keep, 650] and tg.tgemm_last_device_status() == 0
    for b, length in enumerate((n, 650)):
        k = min(length, keep)
        dst = torch.arange(k)
        for h in range(2):
            ref = evict_reference(w[b, h].numpy(), length, keep, 50)
            assert kept[b, h, :k].tolist() == ref and (kept[b, h, k:] == -1).all()
            assert torch.equal(tk[to_table[b].long()[dst // 16], dst % 16, h].double().cpu(), f.k64[b][ref, h])


@pytest.mark.parametrize("kind", ["equal", "special", "negative", "rising"])
def test_evict_weights_of_every_kind(cuda_lib, kind):
    n = 700
    if kind == "equal":
        w = torch.full((1, 2, n), 0.25)
    elif kind == "special":      # NaN, infinities, both zeros, subnormals
        vals = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-42, -1e-42, 1.0, -1.0])
        w = vals[torch.randint(0, len(vals), (1, 2, n), generator=torch.Generator().manual_seed(1))]
    elif kind == "negative":
        w = -torch.rand(1, 2, n, generator=torch.Generator().manual_seed(2))
    else:
        w = torch.arange(n).float().expand(1, 2, n) * 1e-3
    for keep, recent in ((100, 0), (350, 30), (650, 1)):
        run_evict(cuda_lib, [n], 2, 64, 16, "fp16", "16", keep, recent, weights=w, seed=keep)


def test_evict_bad_pages_are_left_out(cuda_lib):
    tg = cuda_lib
    f = Filled(tg, [64], 1, 64, 16, "fp16", seed=20)
    f.table[0, 1] = f.k.shape[0]
    tk, tv = make_pool(2, 16, 1, 64, torch.float16, "pshd", "cuda")
    w = torch.zeros(1, 1, 64)
    w[0, 0, 16:40] = 1 + torch.arange(24)        # the wanted ones: 16 lie on the bad page, 8 do not
    kept = torch.empty(1, 1, 24, dtype=torch.int32, device="cuda")
    tl, tw = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, 1, 24, device="cuda")
    tg.kv_evict(f.cache, f.table, f.lengths, w.cuda(), tg.PagedCache(tk, tv),
                torch.tensor([[1, 0]], dtype=torch.int32).cuda(), kept, tl, tw)
    torch.cuda.synchronize()
    assert tg.tgemm_last_device_status() == CACHE
    assert kept[0, 0].tolist() == list(range(16, 40))
    got = torch.cat([tk[1], tk[0]])[:, 0].float().cpu()
    assert torch.isnan(got[:16]).all() and torch.equal(got[16:24].double(), f.k64[0][32:40, 0]) and torch.isnan(got[24:]).all()
    # A destination past its page list.
    tg.kv_evict(f.cache, f.table, f.lengths, w.cuda(), tg.PagedCache(tk, tv),
                torch.tensor([[1]], dtype=torch.int32).cuda(), kept, tl, tw)
    assert tg.tgemm_last_device_status() == CACHE
