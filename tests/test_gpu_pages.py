"""Bounds of pages, sparse attention by them, and growing, forking, freeing and compacting, against their definitions."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_epilogue_02_gb300 as tg
from kv_helpers import E4M3, TDT, Filled, attend64, attend_bound, score_error, split_e4m3
from page_helpers import Pool, as_list, choose, int32, page_bounds, page_score

pytestmark = pytest.mark.gpu

CACHE_ERROR = 9


def fresh_bounds(cache):
    """Bounds that hold what is not to be read."""
    return tg.PageBounds(torch.full((cache.pages, cache.heads, 2, cache.dim), 99, dtype=torch.int8, device="cuda"),
                         torch.full((cache.pages, cache.heads), float("nan"), device="cuda"))


def keys64(f, page, head):
    """The keys on a page as the values they stand for (e4m3: in fp32), numpy [slots, dim]."""
    if f.ks is None:
        return f.k[page, :, head].double().cpu().numpy()
    return (f.k[page, :, head].float() * f.ks[page, :, head].unsqueeze(-1)).double().cpu().numpy()


def check_bounds(f, bounds, done):
    """The pages `done` have theirs, the others what they had."""
    lo_hi, scale = bounds.bounds.cpu().numpy(), bounds.scale.cpu().numpy()
    for p in range(f.cache.pages):
        for h in range(f.heads):
            if p in done:
                lo, hi, s = page_bounds(keys64(f, p, h))
                assert scale[p, h] == s
                assert (lo_hi[p, h, 0] == lo).all() and (lo_hi[p, h, 1] == hi).all()
            else:
                assert (lo_hi[p, h] == 99).all() and np.isnan(scale[p, h])


BOUNDS = [
    # lengths, new, heads, dim, page, dtype, cache, layout
    ([16, 15, 0, 48, 1], None, 2, 64, 16, "bf16", "16", "pshd"), ([100, 7], [100, 7], 3, 128, 24, "fp16", "16", "phsd"),
    ([64, 200, 33], [1, 150, 0], 1, 256, 32, "bf16", "16", "both"), ([70], [70], 5, 80, 8, "bf16", "16", "pshd"),
    ([130, 1, 77], [130, 1, 50], 2, 128, 24, "bf16", "e4m3", "pshd"), ([65, 9], [65, 9], 4, 64, 16, "fp16", "e4m3", "both"),
    ([90], [90], 1, 256, 10, "bf16", "e4m3", "phsd"), ([12, 3], [12, 3], 2, 96, 1, "fp16", "16", "pshd"),
    ([300], [299], 2, 112, 128, "bf16", "16", "pshd"), ([5], [5], 3, 16, 2, "bf16", "16", "pshd"),
]


@pytest.mark.parametrize("case", BOUNDS, ids=lambda c: "-".join(map(str, c[2:])))
def test_bounds(cuda_lib, case):
    lengths, new, heads, dim, page, dtype, kind, layout = case
    f = Filled(tg, lengths, heads, dim, page, dtype, kind, layout, seed=3)
    bounds = fresh_bounds(f.cache)
    starts = None if new is None else int32([sum(new[:b]) for b in range(len(new) + 1)])
    tg.kv_bounds(f.cache, bounds, f.table, f.lengths, starts=starts)
    torch.cuda.synchronize()
    done = {int(f.table_host[b, i]) for b, n in enumerate(lengths)
            for i in range((n - (new[b] if new else 1)) // page if n else 0, n // page)}
    check_bounds(f, bounds, done)
    assert tg.tgemm_last_device_status() == 0


def test_bounds_of_many_sequences(cuda_lib):
    """More sequences than a block has threads, some without a page done."""
    lengths = [(7 * b) % 40 for b in range(600)]
    f = Filled(tg, lengths, 1, 64, 8, "bf16", seed=5)
    bounds = fresh_bounds(f.cache)
    tg.kv_bounds(f.cache, bounds, f.table, f.lengths, starts=int32([sum(lengths[:b]) for b in range(601)]))
    torch.cuda.synchronize()
    done = {int(f.table_host[b, i]) for b, n in enumerate(lengths) for i in range(n // 8)}
    check_bounds(f, bounds, done)


@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_bounds_of_odd_values(cuda_lib, kind):
    """NaN, infinities, zeros, subnormal and the largest keys; scales that are not finite."""
    f = Filled(tg, [16] * 6, 1, 64, 16, "bf16", kind, seed=6)
    t = [int(f.table_host[b, 0]) for b in range(6)]
    if kind == "16":
        f.k[t[0], 3, 0, 5], f.k[t[0], :, 0, 6] = float("nan"), float("nan")
        f.k[t[1], 2, 0, 7], f.k[t[1], 4, 0, 8] = float("inf"), float("-inf")
        f.k[t[2]] = 0
        f.k[t[3]] = 2.0 ** -133
        f.k[t[4]] = -3.3895313892515355e38
        f.k[t[5], 1, 0, 0] = 2.0 ** -133          # beside keys of order 1: ceil(tiny) is 1
        f.k[t[5], 1:, 0, 1], f.k[t[5], 0, 0, 1] = 0, -2.0 ** -133
    else:
        f.ks[t[0], 3, 0], f.ks[t[1], 2, 0] = float("nan"), float("inf")
        f.ks[t[2]], f.ks[t[3]] = 0, 2.0 ** -140
        f.ks[t[4]] = 1e37
        f.k.view(torch.uint8)[t[5], 4, 0, 9] = 0x7F
    bounds = fresh_bounds(f.cache)
    tg.kv_bounds(f.cache, bounds, f.table, f.lengths)
    torch.cuda.synchronize()
    check_bounds(f, bounds, set(t))


def test_bounds_report_what_is_not_there(cuda_lib):
    f = Filled(tg, [32, 32], 2, 64, 16, "bf16", seed=7)
    f.table[0, 1] = f.cache.pages
    bounds = fresh_bounds(f.cache)
    tg.kv_bounds(f.cache, bounds, f.table, f.lengths, starts=int32([0, 32, 64]))
    torch.cuda.synchronize()
    assert tg.tgemm_last_device_status() == CACHE_ERROR
    check_bounds(f, bounds, {int(f.table_host[0, 0]), int(f.table_host[1, 0]), int(f.table_host[1, 1])})
    for bad in ([-1, 32], [33, 32], [32, 32]):
        starts = int32([0, 40, 20]) if bad == [32, 32] else int32([0, 32, 64])
        tg.kv_bounds(f.cache, fresh_bounds(f.cache), f.table, int32(bad), starts=starts)
        assert tg.tgemm_last_device_status() == CACHE_ERROR


SPARSE = [
    # lengths, heads, group, dim, page, dtype, cache, keep, first, recent, layout
    ([100, 1, 0, 33], 2, 1, 64, 8, "fp16", "16", 5, 1, 2, "pshd"), ([500], 1, 8, 128, 16, "bf16", "16", 7, 0, 1, "phsd"),
    ([300, 77], 3, 5, 80, 10, "bf16", "16", 4, 1, 3, "both"), ([257, 400, 16], 2, 24, 256, 16, "bf16", "16", 9, 0, 4, "pshd"),
    ([900, 30], 4, 9, 128, 16, "fp16", "e4m3", 20, 2, 1, "pshd"), ([640], 2, 2, 96, 1, "fp16", "16", 40, 0, 1, "pshd"),
    ([64, 63], 1, 3, 112, 32, "bf16", "16", 1, 0, 1, "pshd"), ([333], 2, 4, 64, 24, "bf16", "e4m3", 14, 0, 14, "pshd"),
    ([200, 100], 1, 64, 64, 20, "bf16", "16", 3, 0, 1, "pshd"), ([2500, 2499], 1, 2, 64, 4, "fp16", "16", 200, 3, 20, "pshd"),
]


def select(f, q, keep, first, recent, width=None):
    bounds = fresh_bounds(f.cache)
    n = f.lengths_host
    tg.kv_bounds(f.cache, bounds, f.table, f.lengths, starts=int32([sum(n[:b]) for b in range(len(n) + 1)]))
    to_table = torch.full((len(n), f.heads, keep + 3), 55, dtype=torch.int32, device="cuda")
    to_lengths = torch.full((len(n),), 55, dtype=torch.int32, device="cuda")
    tg.kv_select(q, f.cache, bounds, f.table, f.lengths, to_table[:, :, 1:keep + 1], to_lengths, first=first, recent=recent)
    torch.cuda.synchronize()
    assert (to_table[:, :, 0] == 55).all() and (to_table[:, :, keep + 1:] == 55).all()
    return to_table[:, :, 1:keep + 1], to_lengths, bounds


def selection(f, q, keep, first, recent):
    """By the definition: positions' pages of each sequence and head, and lengths."""
    lists, lengths = [], []
    group = q.shape[1] // f.heads
    for b, n in enumerate(f.lengths_host):
        count = -(-n // f.page)
        rows = []
        for h in range(f.heads):
            queries = q[b, h * group:(h + 1) * group].double().cpu().numpy()
            scores = [page_score(queries, *page_bounds(keys64(f, int(f.table_host[b, i]), h))) if i < n // f.page else 0.0
                      for i in range(count)] if count > keep else [0.0] * count
            rows.append(choose(scores, keep, first, recent))
        lists.append(rows)
        lengths.append(n - (count - min(count, keep)) * f.page)
    return lists, lengths


@pytest.mark.parametrize("case", SPARSE, ids=lambda c: "-".join(map(str, c[1:])))
def test_selection_and_attention(cuda_lib, case):
    lengths, heads, group, dim, page, dtype, kind, keep, first, recent, layout = case
    f = Filled(tg, lengths, heads, dim, page, dtype, kind, layout, seed=11)
    g = torch.Generator().manual_seed(2)
    q = (torch.randn(len(lengths), heads * group, dim, generator=g) * 2).to(TDT[dtype]).cuda()
    to_table, to_lengths, _ = select(f, q, keep, first, recent)
    lists, want = selection(f, q, keep, first, recent)
    assert as_list(to_lengths) == want
    got = as_list(to_table)
    for b in range(len(lengths)):
        for h in range(heads):
            pages = [int(f.table_host[b, i]) for i in lists[b][h]]
            assert got[b][h] == pages + [-1] * (keep - len(pages)), (b, h)
    # Attention over the lists, and its accumulated weights by their positions.
    o = torch.full_like(q, 3.0)
    w = torch.ones(len(lengths), heads, keep * page, device="cuda")
    lists_table = to_table.contiguous()
    tg.attention_decode(q, f.cache, lists_table, to_lengths, o, weights=w)
    o2 = torch.empty_like(q)
    tg.attention_decode(q, f.cache, to_table, to_lengths, o2,                     # strided lists, a workspace of the caller's
                        workspace=tg.attention_decode_workspace(q, f.cache, to_table))
    torch.cuda.synchronize()
    assert torch.equal(o, o2)
    p_dtype = "fp16" if kind == "e4m3" else dtype
    for b, n in enumerate(lengths):
        for h in range(heads):
            pos = torch.tensor([i * page + s for i in lists[b][h] for s in range(page) if i * page + s < n], dtype=torch.long)
            rows = slice(h * group, (h + 1) * group)
            k, v = f.k64[b][:, h:h + 1], f.v64[b][:, h:h + 1]
            o64, p, mag, reach, top = attend64(q[b, rows].cpu(), k, v, dim ** -0.5, keep=pos)
            bound = attend_bound(o64, mag, reach, top, len(pos), dim, dtype, p_dtype, 0.0)
            assert ((o[b, rows].double().cpu() - o64).abs() <= bound).all()
            if len(pos):
                grown = w[b, h, :len(pos)].double().cpu() - 1
                assert (grown - p[:, pos].sum(0)).abs().max() <= group * (1e-3 if dtype == "bf16" else 1e-3)
            assert (w[b, h, len(pos):] == 1).all()
    assert tg.tgemm_last_device_status() == 0


def test_lists_that_the_heads_share_are_as_before(cuda_lib):
    """A list for each head that is the same for all gives the bits of one shared list."""
    f = Filled(tg, [700, 33, 0, 2000], 3, 128, 16, "bf16", seed=12)
    q = torch.randn(4, 12, 128, device="cuda").bfloat16()
    a, b = torch.empty_like(q), torch.empty_like(q)
    tg.attention_decode(q, f.cache, f.table, f.lengths, a, window=900, cap=20.0)
    tg.attention_decode(q, f.cache, f.table.unsqueeze(1).expand(-1, 3, -1).contiguous(), f.lengths, b, window=900, cap=20.0)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_one_head_with_any_stride(cuda_lib):
    """A size of 1 may have any stride."""
    f = Filled(tg, [100, 3], 1, 64, 16, "fp16", seed=12)
    q = torch.randn(2, 4, 64, device="cuda").half()
    a, b = torch.empty_like(q), torch.empty_like(q)
    tg.attention_decode(q, f.cache, f.table, f.lengths, a)
    tg.attention_decode(q, f.cache, f.table.as_strided((2, 1, f.table.shape[1]), (f.table.stride(0), 1, 1)), f.lengths, b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_ties_go_to_the_lowest_position(cuda_lib):
    """Pages of equal keys, queries of zeros: equal scores everywhere."""
    f = Filled(tg, [400], 2, 64, 8, "fp16", seed=13)
    f.k.zero_()
    for value in (0.0, 1.0):
        q = torch.full((1, 4, 64), value, dtype=torch.float16, device="cuda")
        to_table, _, _ = select(f, q, 10, 1, 2)
        want = [int(f.table_host[0, i]) for i in [0] + list(range(1, 8)) + [48, 49]]
        assert as_list(to_table) == [[want] * 2]


def test_extreme_queries_and_keys(cuda_lib):
    """Whole numbers at the ends of their range over the longest rows keep their sums exact; NaN counts as zero, an
    infinity as the largest number."""
    f = Filled(tg, [320], 1, 256, 16, "bf16", seed=14)
    f.k.copy_(torch.where(f.k > 0, 127.0, -127.0))
    for i in range(20):
        f.k[int(f.table_host[0, i]), 0, 0, i] = 126.0           # pages that differ by one in one channel
    q = torch.where(torch.randn(1, 64, 256, device="cuda") > 0, 127.0, -127.0).bfloat16()
    q[0, 1, 3], q[0, 2, 5], q[0, 3] = float("nan"), float("inf"), 0
    to_table, _, _ = select(f, q, 6, 0, 1)
    lists, _ = selection(f, q, 6, 0, 1)
    assert as_list(to_table)[0][0] == [int(f.table_host[0, i]) for i in lists[0][0]]


@pytest.mark.parametrize("pages,batch,dim,group", [
    (3000, 1, 64, 3), (9000, 2, 64, 3), (17000, 1, 64, 3), (600, 40, 64, 3), (5000, 1, 128, 24), (700, 100, 128, 8), (4000, 2, 256, 8),
    (131072, 1, 256, 64), (131072, 1, 64, 1),
])
def test_long_lists(cuda_lib, pages, batch, dim, group):
    """One block and clusters, more pages than one block has room for, the longest list with the most heads."""
    g = torch.Generator().manual_seed(15)
    heads, keep = 2 if pages < 100000 else 1, 100
    cache = tg.PagedCache(*(torch.zeros(pages, 1, heads, dim, dtype=torch.float16, device="cuda") for _ in range(2)))
    bounds = tg.PageBounds(torch.randint(-127, 128, (pages, heads, 2, dim), dtype=torch.int8, generator=g).cuda(),
                           (2.0 ** torch.randint(-3, 1, (pages, heads), generator=g)).cuda())
    table = torch.stack([torch.randperm(pages, generator=g) for _ in range(batch)]).to(torch.int32).cuda()
    lengths = torch.randint(1, pages + 1, (batch,), generator=g).to(torch.int32)
    lengths[0] = pages
    q = torch.randint(-127, 128, (batch, heads * group, dim), generator=g).half().cuda()
    q[..., 0] = 127                                              # the power of two is 1
    to_table, to_lengths = torch.empty(batch, heads, keep, dtype=torch.int32, device="cuda"), torch.empty_like(lengths).cuda()
    tg.kv_select(q, cache, bounds, table, lengths.cuda(), to_table, to_lengths, first=2, recent=3)
    torch.cuda.synchronize()
    for b in range(batch):
        n = int(lengths[b])
        at = table[b, :n].long()
        lo, hi = bounds.bounds[at, :, 0].double(), bounds.bounds[at, :, 1].double()
        for h in range(heads):
            s = torch.full((n,), -float("inf"), dtype=torch.float64, device="cuda")
            for z in q[b, h * group:(h + 1) * group].double():
                # bounds of any order: the lower one counts where z < 0
                s = torch.maximum(s, lo[:, h] @ z.clamp(max=0) + hi[:, h] @ z.clamp(min=0))
            kept = choose((s * bounds.scale[at, h].double()).tolist(), keep, 2, 3)
            assert as_list(to_table[b, h]) == as_list(at[kept]) + [-1] * (keep - len(kept))


def test_selection_reports_bad_pages(cuda_lib):
    f = Filled(tg, [160], 1, 64, 16, "bf16", seed=16)
    q = torch.randn(1, 2, 64, device="cuda").bfloat16()
    _, _, bounds = select(f, q, 4, 0, 1)
    f.table[0, 3], f.table[0, 5] = -7, f.cache.pages
    to_table, to_lengths = torch.empty(1, 1, 8, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    tg.kv_select(q, f.cache, bounds, f.table, f.lengths, to_table, to_lengths)
    assert tg.tgemm_last_device_status() == CACHE_ERROR
    kept = as_list(to_table)[0][0]
    assert -7 not in kept and f.cache.pages not in kept and len(set(kept)) == 8          # the others score higher
    for n in (-1, 161):
        tg.kv_select(q, f.cache, bounds, f.table, int32([n]), to_table, to_lengths)
        assert tg.tgemm_last_device_status() == CACHE_ERROR
        assert as_list(to_lengths) == [0 if n < 0 else 128]


# ---------------------------------------------------------------- pages
class Held:
    """A cache with sequences in some of its pages, on the GPU and as lists."""

    def __init__(self, lengths, page, pages, heads=2, dim=64, kind="16", layout="pshd", seed=0, width=None, shared=()):
        g = torch.Generator().manual_seed(seed)
        ctype = E4M3 if kind == "e4m3" else torch.bfloat16
        shape = (pages, heads, page, dim) if layout == "phsd" else (pages, page, heads, dim)
        pools = [torch.randn(shape, generator=g).cuda().to(ctype) for _ in range(2)]
        if layout == "phsd":
            pools = [t.transpose(1, 2) for t in pools]
        self.scales = [torch.rand(pages, page, heads, generator=g).cuda() for _ in range(2)] if kind == "e4m3" else [None, None]
        self.cache = tg.PagedCache(*pools, *self.scales)
        need = [-(-n // page) for n in lengths]
        order = torch.randperm(pages, generator=g).tolist()
        self.width = width or max(need) + 2
        self.table, at = [], 0
        for n in need:
            self.table.append(order[at:at + n] + [-9] * (self.width - n))
            at += n
        self.lengths = list(lengths)
        for b in shared:                               # a sequence that holds another's full pages
            full = lengths[b] // page
            self.table.append(self.table[b][:full] + [-9] * (self.width - full))
            self.lengths.append(full * page)
        uses = [0] * pages
        for row, n in zip(self.table, self.lengths):
            for i in range(-(-n // page)):
                uses[row[i]] += 1
        self.pool = Pool(uses, page, self.width)
        self.page, self.g = page, g
        self.d_uses, self.d_table, self.d_lengths = int32(uses), int32(self.table), int32(self.lengths)

    def parts(self):
        return [t for t in (self.cache.k, self.cache.v, *self.scales) if t is not None]

    def images(self):
        return [t.float().cpu() for t in self.parts()]

    def check(self, table=None, lengths=None, uses=None):
        torch.cuda.synchronize()
        assert as_list(self.d_uses if uses is None else uses) == self.pool.uses
        assert as_list(self.d_table if table is None else table) == self.table
        assert as_list(self.d_lengths if lengths is None else lengths) == self.lengths


@pytest.mark.parametrize("page", [1, 7, 16])
def test_grow(cuda_lib, page):
    h = Held([0, 5, 16, 33, 1], page, 200, width=120 // page + 8)
    for tokens in ([1, 1, 1, 1, 1], [0, 30, 0, 17, 64], [1, 1, 1, 1, 1]):
        given = None if tokens == [1] * 5 else int32(tokens)
        tg.kv_grow(h.cache, h.d_uses, h.d_table, h.d_lengths, tokens=given)
        h.pool.grow(h.table, h.lengths, tokens)
        h.check()
    assert tg.tgemm_last_device_status() == 0


def test_grow_of_many(cuda_lib):
    """More sequences than a block has threads, a pool of several rounds, pages by the hundred for some."""
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 60, (1500,), generator=g).tolist()
    h = Held(lengths, 16, 30000, heads=1, dim=16, width=230, seed=4)
    for i in range(2):
        tokens = torch.randint(0, 50, (1500,), generator=g).tolist()
        tokens[7 + i], tokens[1200 + i] = 3000, 2500
        tg.kv_grow(h.cache, h.d_uses, h.d_table, h.d_lengths, tokens=int32(tokens))
        h.pool.grow(h.table, h.lengths, tokens)
        h.check()


def test_grow_refuses_on_the_device(cuda_lib):
    """No room in the list, none in the pool, bad lengths and counts: reported, the sequence as it was."""
    h = Held([16, 16, 16, 16], 16, 7, width=3)                  # three pages left
    for tokens, ok in (([1, 33, -1, 0], False), ([16, 17, 1, 0], False)):
        tg.kv_grow(h.cache, h.d_uses, h.d_table, h.d_lengths, tokens=int32(tokens))
        before = [row[:] for row in h.table]
        h.pool.grow(h.table, h.lengths, tokens)
        torch.cuda.synchronize()
        assert as_list(h.d_uses) == h.pool.uses and as_list(h.d_lengths) == h.lengths
        got = as_list(h.d_table)
        for b, n in enumerate(h.lengths):                        # what is past a length may have been written
            assert got[b][:-(-n // 16)] == h.table[b][:-(-n // 16)]
        assert tg.tgemm_last_device_status() == CACHE_ERROR
        h.table = before if not ok else h.table
        h.table = got
    h.d_lengths[1] = -4
    tg.kv_grow(h.cache, h.d_uses, h.d_table, h.d_lengths, tokens=int32([0, 1, 0, 0]))
    assert tg.tgemm_last_device_status() == CACHE_ERROR and as_list(h.d_lengths)[1] == -4


FORKS = [
    ([37, 5, 32, 0], [0, 0, 2, 1, 3, -1, 0], 16, "16", "pshd"), ([100, 64], [1, 0, 0, 1], 24, "e4m3", "pshd"),
    ([9], [0] * 40, 4, "16", "phsd"), ([50, 3], [1, 1, 0], 1, "16", "pshd"), ([200], [0, 0], 128, "e4m3", "phsd"),
]


@pytest.mark.parametrize("case", FORKS, ids=lambda c: f"{len(c[1])}-{c[2]}-{c[3]}-{c[4]}")
@pytest.mark.parametrize("same", [False, True])
def test_fork_and_free(cuda_lib, case, same):
    """Children in a table of their own, and in other rows of the parents'."""
    lengths, parents, page, kind, layout = case
    children = len(parents)
    h = Held(lengths, page, 260, kind=kind, layout=layout, seed=5)
    if same:
        rows = [[-9] * h.width for _ in range(children)]
        whole, all_lengths = int32(h.table + rows), int32(h.lengths + [0] * children)
        h.d_table, to = whole[:len(lengths)], whole[len(lengths):]
        h.d_lengths, to_lengths = all_lengths[:len(lengths)], all_lengths[len(lengths):]
    else:
        to, to_lengths = torch.full((children, h.width), -9, dtype=torch.int32, device="cuda"), int32([0] * children)
    for _ in range(2):
        want = h.images()
        tg.kv_fork(h.cache, h.d_uses, h.d_table, h.d_lengths, int32(parents), to, to_lengths)
        to_host, n_host = [[-9] * h.width for _ in range(children)], [0] * children
        for a, z, rows in h.pool.fork(h.table, h.lengths, parents, to_host, n_host):
            for t in want:
                t[z, :rows] = t[a, :rows]
        h.check()
        assert as_list(to) == to_host and as_list(to_lengths) == n_host
        assert all(torch.equal(a, b) for a, b in zip(h.images(), want))
        tg.kv_free(h.cache, h.d_uses, to, to_lengths)
        h.pool.free(to_host, n_host)
        h.check()
        assert as_list(to_lengths) == n_host
        to.fill_(-9)
    assert tg.tgemm_last_device_status() == 0


def test_fork_refuses_on_the_device(cuda_lib):
    """Parents that are not there, a list without room, a pool without pages."""
    h = Held([20, 40], 16, 7, seed=6)                            # two pages left
    parents = [5, -3, 0, 1, 0]                                   # 0, 1 and 0 want a page each
    to, to_lengths = torch.full((5, h.width), -9, dtype=torch.int32, device="cuda"), int32([0] * 5)
    want = h.images()
    tg.kv_fork(h.cache, h.d_uses, h.d_table, h.d_lengths, int32(parents), to, to_lengths)
    to_host, n_host = [[-9] * h.width for _ in range(5)], [0] * 5
    for a, z, rows in h.pool.fork(h.table, h.lengths, parents, to_host, n_host):
        for t in want:
            t[z, :rows] = t[a, :rows]
    h.check()
    assert h.pool.error and tg.tgemm_last_device_status() == CACHE_ERROR
    assert as_list(to) == to_host and as_list(to_lengths) == n_host == [0, 0, 20, 40, 16]
    assert all(torch.equal(a, b) for a, b in zip(h.images(), want))
    short, short_lengths = torch.full((1, 2), -9, dtype=torch.int32, device="cuda"), int32([0])
    tg.kv_fork(h.cache, h.d_uses, h.d_table, h.d_lengths, int32([1]), short, short_lengths)
    h.check()
    assert tg.tgemm_last_device_status() == CACHE_ERROR and as_list(short_lengths) == [0]


def test_free_reports_pages_that_are_free(cuda_lib):
    h = Held([30, 20], 16, 8, seed=7)
    h.d_uses[h.table[1][1]] = 0
    h.d_table[0, 0] = 8
    tg.kv_free(h.cache, h.d_uses, h.d_table, h.d_lengths)
    torch.cuda.synchronize()
    assert tg.tgemm_last_device_status() == CACHE_ERROR
    uses = as_list(h.d_uses)
    assert uses[h.table[1][1]] == 0 and uses[h.table[1][0]] == 0 and uses[h.table[0][1]] == 0 and uses[h.table[0][0]] == 1
    assert as_list(h.d_lengths) == [0, 0]


COMPACTS = [
    ([37, 5, 0, 32], 16, 30, "16", "pshd", (0,)), ([100, 64, 3], 24, 60, "e4m3", "pshd", (0, 1)), ([9, 8], 4, 5, "16", "phsd", ()),
    ([300, 200, 77], 1, 2500, "16", "pshd", (2,)), ([500, 1], 64, 40, "e4m3", "phsd", (0, 0)), ([0], 16, 9, "16", "pshd", ()),
    ([1000, 3000], 8, 9000, "16", "pshd", (1,)),
]


@pytest.mark.parametrize("case", COMPACTS, ids=lambda c: f"{sum(c[0])}-{c[1]}-{c[2]}-{c[3]}-{c[4]}")
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("with_bounds", [False, True])
def test_compact(cuda_lib, case, in_place, with_bounds):
    lengths, page, pages, kind, layout, shared = case
    h = Held(lengths, page, pages, kind=kind, layout=layout, seed=8, shared=shared)
    bounds = None
    if with_bounds:
        bounds = tg.PageBounds(torch.randint(-127, 128, (pages, 2, 2, 64), dtype=torch.int8, generator=h.g).cuda(),
                               torch.rand(pages, 2, generator=h.g).cuda())
    want = h.images() + ([bounds.bounds.cpu(), bounds.scale.cpu()] if bounds else [])
    to, to_uses = (h.d_table, h.d_uses) if in_place else (torch.full_like(h.d_table, -9), torch.full_like(h.d_uses, 77))
    in_use = int32([0])
    for round_ in range(2):                                      # nothing moves the second time
        tg.kv_compact(h.cache, h.d_uses, h.d_table, h.d_lengths, to, to_uses, in_use, bounds=bounds)
        moves, n = h.pool.compact(h.table, h.lengths)
        for a, z in moves.items():
            for t in want:
                t[z] = t[a]
        h.check(table=to, uses=to_uses)
        assert as_list(in_use) == [n] and (round_ == 0 or not moves)
        got = h.images() + ([bounds.bounds.cpu(), bounds.scale.cpu()] if bounds else [])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        h.d_table, h.d_uses = to, to_uses
        if not in_place:
            to, to_uses = torch.full_like(to, -9), torch.full_like(to_uses, 77)
    assert tg.tgemm_last_device_status() == 0


def test_compact_reports_pages_that_nothing_counts(cuda_lib):
    h = Held([40, 40], 16, 20, seed=9)
    high = max(h.table[0][:3])
    h.d_uses[high] = 0
    h.pool.uses[high] = 0
    h.d_table[1, 2] = 20
    to, to_uses, in_use = torch.full_like(h.d_table, -9), torch.empty_like(h.d_uses), int32([0])
    tg.kv_compact(h.cache, h.d_uses, h.d_table, h.d_lengths, to, to_uses, in_use)
    torch.cuda.synchronize()
    assert tg.tgemm_last_device_status() == CACHE_ERROR and as_list(in_use) == [5]
    moves, _ = h.pool.compact([], [])
    assert as_list(to_uses) == h.pool.uses and as_list(to)[1][2] == 20


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("stream", [False, True])
def test_serving_loop(cuda_lib, kind, stream):
    """Prompts, steps with rotation, bounds and sparse attention, children, freeing and compaction, one call after another
    without a synchronisation; every step's output against a plain computation from what was appended."""
    heads, group, dim, page, keep, slots, width, pages = 2, 2, 64, 8, 5, 4, 12, 60
    ctype = E4M3 if kind == "e4m3" else torch.bfloat16
    side = torch.cuda.Stream() if stream else None
    g = torch.Generator().manual_seed(21)
    pools = [torch.zeros(pages, page, heads, dim, device="cuda").to(ctype) for _ in range(2)]
    scales = [torch.zeros(pages, page, heads, device="cuda") for _ in range(2)] if kind == "e4m3" else [None, None]
    cache = tg.PagedCache(*pools, *scales)
    bounds = tg.PageBounds(torch.zeros(pages, heads, 2, dim, dtype=torch.int8, device="cuda"), torch.ones(pages, heads, device="cuda"))
    uses, in_use = torch.zeros(pages, dtype=torch.int32, device="cuda"), int32([0])
    table, lengths = torch.zeros(slots, width, dtype=torch.int32, device="cuda"), torch.zeros(slots, dtype=torch.int32, device="cuda")
    rotary = tg.Rotary([100.0 ** (-i / 32) for i in range(32)])
    w = [(1 + 0.1 * torch.randn(dim, generator=g)).bfloat16().cuda() for _ in range(2)]
    to_table = torch.zeros(slots, heads, keep, dtype=torch.int32, device="cuda")
    to_lengths = torch.zeros(slots, dtype=torch.int32, device="cuda")
    rows = [[] for _ in range(slots)]                       # (k, v) as appended, [heads, dim] each
    checks = []
    torch.cuda.synchronize()

    def step(counts):
        """counts[b] new tokens of each sequence."""
        n = sum(counts)
        q = (torch.randn(n, heads * group, dim, generator=g) * 2).bfloat16().cuda()
        k, v = (torch.randn(n, heads, dim, generator=g).bfloat16().cuda() for _ in range(2))
        starts = int32([sum(counts[:b]) for b in range(slots + 1)])
        at = [len(rows[b]) + i for b in range(slots) for i in range(counts[b])]
        positions = int32([at])
        torch.cuda.synchronize()
        tg.kv_grow(cache, uses, table, lengths, tokens=int32(counts), stream=side)
        tg.qk_norm_rope(q, k, positions, rotary, q, k, q_weight=w[0], k_weight=w[1], stream=side)
        tg.kv_append(cache, k, v, table, lengths, starts=starts, stream=side)
        tg.kv_bounds(cache, bounds, table, lengths, starts=starts, stream=side)
        if side:
            side.synchronize()
        torch.cuda.synchronize()
        for i, b in enumerate(b for b in range(slots) for _ in range(counts[b])):
            rows[b].append((k[i].clone(), v[i].clone()))
        last = torch.zeros(slots, heads * group, dim, dtype=torch.bfloat16, device="cuda")
        for b in range(slots):
            if counts[b]:
                last[b] = q[sum(counts[:b + 1]) - 1]
        out, full = torch.empty_like(last), torch.empty_like(last)
        torch.cuda.synchronize()
        tg.kv_select(last, cache, bounds, table, lengths, to_table, to_lengths, first=1, recent=2, stream=side)
        tg.attention_decode(last, cache, to_table, to_lengths, out, stream=side)
        tg.attention_decode(last, cache, table, lengths, full, stream=side)
        if side:
            side.synchronize()
        torch.cuda.synchronize()
        chosen = as_list(to_table)
        lists = as_list(table)
        for b in range(slots):
            n = len(rows[b])
            assert int(lengths[b]) == n
            for h in range(heads):
                pages_kept = [lists[b].index(p) for p in chosen[b][h] if p >= 0]
                pos = [i * page + s for i in pages_kept for s in range(page) if i * page + s < n]
                checks.append((last[b, h * group:(h + 1) * group], [rows[b][i] for i in pos], h, out[b, h * group:(h + 1) * group]))
                checks.append((last[b, h * group:(h + 1) * group], list(rows[b]), h, full[b, h * group:(h + 1) * group]))

    step([50, 9, 0, 23])
    for _ in range(9):
        step([1, 1, 0, 1])
    # Sequence 1 ends, 1 and 2 become children of 0.
    children, child_lengths = table[1:3], lengths[1:3]
    tg.kv_free(cache, uses, children, child_lengths, stream=side)
    tg.kv_fork(cache, uses, table, lengths, int32([0, 0]), children, child_lengths, stream=side)
    rows[1], rows[2] = list(rows[0]), list(rows[0])
    for _ in range(4):
        step([1, 1, 1, 1])
    tg.kv_free(cache, uses, table[:1], lengths[:1], stream=side)
    rows[0] = []
    tg.kv_compact(cache, uses, table, lengths, table, uses, in_use, bounds=bounds, stream=side)
    if side:
        side.synchronize()
    torch.cuda.synchronize()
    assert int(in_use) == int((uses > 0).sum()) and (uses[int(in_use):] == 0).all()
    for _ in range(10):
        step([3, 1, 1, 1])
    assert tg.tgemm_last_device_status() == 0
    for q, kept, h, got in checks:
        if not kept:
            assert (got == 0).all()
            continue
        k, v = (torch.stack([r[i][h] for r in kept]).cpu() for i in range(2))
        if kind == "e4m3":                                       # (on the CPU: a GPU's tensor / 448 is a product)
            k, v = (e.float().double() * s.double().unsqueeze(-1) for e, s in (split_e4m3(x) for x in (k, v)))
        k, v, q, got = k.double(), v.double(), q.cpu(), got.cpu()
        p = torch.softmax(k @ q.double().T * dim ** -0.5, 0)
        want = p.T @ v
        # bf16's half step of the output; weights off by 2^-16, their exponents by less than 2^-14
        assert (got.double() - want).abs().max() <= 2.0 ** -8 * want.abs().max() + 2.0 ** -12 * v.abs().max()


def test_calls_in_a_graph(cuda_lib):
    """One step captured and replayed: it follows the lengths and pages that it finds."""
    def new():
        h = Held([30, 17, 1], 8, 80, seed=30, width=20)
        g = torch.Generator().manual_seed(31)
        bounds = tg.PageBounds(torch.zeros(80, 2, 2, 64, dtype=torch.int8, device="cuda"), torch.ones(80, 2, device="cuda"))
        tg.kv_bounds(h.cache, bounds, h.d_table, h.d_lengths, starts=int32([0, 30, 47, 48]))
        s = dict(h=h, bounds=bounds, q=torch.randn(3, 4, 64, generator=g).bfloat16().cuda(),
                 k=torch.randn(3, 2, 64, generator=g).bfloat16().cuda(), v=torch.randn(3, 2, 64, generator=g).bfloat16().cuda(),
                 to=torch.zeros(3, 2, 3, dtype=torch.int32, device="cuda"), n=torch.zeros(3, dtype=torch.int32, device="cuda"),
                 o=torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda"), child=torch.zeros(2, 20, dtype=torch.int32, device="cuda"),
                 child_n=torch.zeros(2, dtype=torch.int32, device="cuda"), parents=int32([0, 2]),
                 moved=torch.zeros(3, 20, dtype=torch.int32, device="cuda"), in_use=int32([0]), left=torch.zeros(80, dtype=torch.int32, device="cuda"))
        s["ws"] = tg.attention_decode_workspace(s["q"], h.cache, s["to"])
        s["cws"] = tg.kv_compact_workspace(h.cache)
        s["rotary"] = tg.Rotary([0.5] * 32)
        return s

    def step(s):
        h = s["h"]
        tg.kv_free(h.cache, h.d_uses, s["child"], s["child_n"])
        tg.kv_grow(h.cache, h.d_uses, h.d_table, h.d_lengths)
        tg.qk_norm_rope(s["q"], s["k"], h.d_lengths, s["rotary"], s["q"], s["k"], shift=-1)
        tg.kv_append(h.cache, s["k"], s["v"], h.d_table, h.d_lengths)
        tg.kv_bounds(h.cache, s["bounds"], h.d_table, h.d_lengths)
        tg.kv_select(s["q"], h.cache, s["bounds"], h.d_table, h.d_lengths, s["to"], s["n"])
        tg.attention_decode(s["q"], h.cache, s["to"], s["n"], s["o"], workspace=s["ws"])
        tg.kv_fork(h.cache, h.d_uses, h.d_table, h.d_lengths, s["parents"], s["child"], s["child_n"])

    def outputs(s):
        h = s["h"]
        return h.parts() + [h.d_uses, h.d_table, h.d_lengths, s["to"], s["n"], s["o"], s["child"], s["child_n"], s["bounds"].bounds,
                            s["bounds"].scale]

    a, b = new(), new()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for i in range(40):
        a["parents"].copy_(int32([i % 3, (i + 1) % 3]))
        b["parents"].copy_(a["parents"])
        graph.replay()
        step(b)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outputs(a), outputs(b)))
    assert tg.tgemm_last_device_status() == 0
    for s in (a, b):
        h = s["h"]
        tg.kv_compact(h.cache, h.d_uses, torch.cat([h.d_table, s["child"]]), torch.cat([h.d_lengths, s["child_n"]]),
                      torch.zeros(5, 20, dtype=torch.int32, device="cuda"), s["left"], s["in_use"], workspace=s["cws"])
    torch.cuda.synchronize()
    assert torch.equal(a["left"], b["left"]) and torch.equal(a["in_use"], b["in_use"])
    assert all(torch.equal(x, y) for x, y in zip(a["h"].parts(), b["h"].parts()))


def test_empty_batches_and_pools(cuda_lib):
    cache = tg.PagedCache(*(torch.zeros(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    bounds = tg.PageBounds(torch.zeros(0, 2, 2, 64, dtype=torch.int8, device="cuda"), torch.zeros(0, 2, device="cuda"))
    uses = torch.zeros(0, dtype=torch.int32, device="cuda")
    for batch in (0, 2):
        table, lengths = torch.zeros(batch, 3, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.int32, device="cuda")
        q = torch.zeros(batch, 4, 64, dtype=torch.bfloat16, device="cuda")
        to, n, in_use = torch.zeros(batch, 2, 2, dtype=torch.int32, device="cuda"), torch.zeros_like(lengths), int32([5])
        tg.kv_bounds(cache, bounds, table, lengths)
        tg.kv_select(q, cache, bounds, table, lengths, to, n)
        tg.attention_decode(q, cache, to, n, q.clone())
        tg.kv_grow(cache, uses, table, lengths, tokens=torch.zeros_like(lengths))
        tg.kv_free(cache, uses, table, lengths)
        tg.kv_fork(cache, uses, table, lengths, torch.full_like(lengths, -1), table.clone(), n)
        tg.kv_compact(cache, uses, table, lengths, table, uses, in_use)
        torch.cuda.synchronize()
        assert as_list(in_use) == [0]
    status = tg.tgemm_last_device_status()
    assert status == 0, status
    tg.kv_grow(cache, uses, table, lengths)
    assert tg.tgemm_last_device_status() == CACHE_ERROR and as_list(lengths) == [0, 0]


def test_debug_build_finds_nothing(cuda_lib):
    from gemm_epilogue_02_gb300 import _binding
    release, dbg = _binding._lib, tg.load_debug()
    assert dbg.tgemm_debug_last_check() == 0
    _binding._lib = dbg
    try:
        for case in BOUNDS[:3] + BOUNDS[4:6]:
            test_bounds.__wrapped__(None, case) if hasattr(test_bounds, "__wrapped__") else test_bounds(None, case)
        for case in SPARSE[:5]:
            test_selection_and_attention(None, case)
        for case in FORKS[:3]:
            test_fork_and_free(None, case, False)
        for case in COMPACTS[:4]:
            test_compact(None, case, False, True)
        torch.cuda.synchronize()
        assert dbg.tgemm_last_device_status() == 0 and dbg.tgemm_debug_last_check() == 0
    finally:
        _binding._lib = release


def test_example_runs(cuda_lib):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_samples.py")
    spec = importlib.util.spec_from_file_location("decode_samples", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer, used, status = example.main(steps=20)
    assert status == 0
    # Prompts of 300 and 77; 20 and 20 steps; one more after the compaction.  Two sequences that began again at the third's 320.
    assert as_list(layer.lengths) == [341, 118, 341, 341, 341, 341, 118, 118]
    uses, table, size = as_list(layer.uses), as_list(layer.table), 16
    held = [0] * len(uses)
    for row, n in zip(table, as_list(layer.lengths)):
        for p in row[:-(-n // size)]:
            held[p] += 1
    assert uses == held
    assert used == sum(u > 0 for u in held) - sum(n % size == 1 for n in as_list(layer.lengths))
    # 300 positions are 18 full pages, 77 are 4: held by the prompt and its continuations alike.
    assert all(table[b][:18] == table[0][:18] for b in (2, 3, 4, 5)) and all(table[b][:4] == table[1][:4] for b in (6, 7))


@pytest.mark.parametrize("group", [1, 4, 9])
def test_weights_over_lists_that_differ(cuda_lib, group):
    """A page that is not in the pool, in the list of one head: the weights of that head there stay, those of the others
    grow by their attention, in the first head's list and in another's."""
    n, heads, dim, page = 150, 3, 64, 16
    f = Filled(tg, [n, n], heads, dim, page, "bf16", seed=40, extra=9)
    q = torch.randn(2, heads * group, dim, device="cuda").bfloat16()
    lists = f.table.unsqueeze(1).expand(-1, heads, -1).contiguous()
    lists[0, 0, 2], lists[1, 1, 4], lists[1, 2, 0] = f.cache.pages, -1, 2 ** 30
    gone = {(0, 0): 2, (1, 1): 4, (1, 2): 0}
    o, w = torch.empty_like(q), torch.full((2, heads, n + 5), 2.0, device="cuda")
    ws = tg.attention_decode_workspace(q, f.cache, lists, weights=True)
    for round_ in range(2):                                       # the second finds the first one's scores in the workspace
        tg.attention_decode(q, f.cache, lists, f.lengths, o, weights=w, workspace=ws)
        assert tg.tgemm_last_device_status() == CACHE_ERROR
        for b in range(2):
            for h in range(heads):
                bad = gone.get((b, h))
                pos = torch.tensor([j for j in range(n) if j // page != bad])
                rows = slice(h * group, (h + 1) * group)
                o64, p, mag, reach, top = attend64(q[b, rows].cpu(), f.k64[b][:, h:h + 1], f.v64[b][:, h:h + 1], dim ** -0.5, keep=pos)
                bound = attend_bound(o64, mag, reach, top, len(pos), dim, "bf16", "bf16", 0.0)
                assert ((o[b, rows].double().cpu() - o64).abs() <= bound).all()
                # a weight of p: its exponent's error and that of the sum below it, the sum's roundings, two exponentials and
                # a division of 2^-22 each; then the group's sum and what is there, below group and 2 + 2 group
                e = 2 * score_error(reach, dim, 0.0) + (n + 64) * 2.0 ** -24 + 2.0 ** -20
                room = (p * e.unsqueeze(-1)).sum(0) + (group ** 2 + 2 * group + 2) * 2.0 ** -24
                grown = w[b, h, :n].double().cpu() - 2
                assert ((grown - (round_ + 1) * p.sum(0)).abs() <= (round_ + 1) * room).all(), (b, h)
                if bad is not None:
                    assert (w[b, h, bad * page:(bad + 1) * page] == 2).all()
                assert (w[b, h, n:] == 2).all()


@pytest.mark.parametrize("children", [2, 40])
def test_fork_leaves_bad_lengths_out(cuda_lib, children):
    """A parent's length below 0 or past what its list holds: the child is empty, no count changes."""
    for bad in (-1, 49, 2 ** 31 - 1):
        h = Held([48, 20], 16, 60, seed=41, width=3)
        h.d_lengths[0] = bad
        parents = [0, 1] * (children // 2)
        to, to_lengths = torch.full((children, 3), -9, dtype=torch.int32, device="cuda"), int32([5] * children)
        want = h.images()
        tg.kv_fork(h.cache, h.d_uses, h.d_table, h.d_lengths, int32(parents), to, to_lengths)
        to_host, n_host = [[-9] * 3 for _ in range(children)], [0] * children
        for a, z, rows in h.pool.fork(h.table, h.lengths, [-1 if p == 0 else p for p in parents], to_host, n_host):
            for t in want:
                t[z, :rows] = t[a, :rows]
        torch.cuda.synchronize()
        assert tg.tgemm_last_device_status() == CACHE_ERROR
        assert as_list(h.d_uses) == h.pool.uses and as_list(to_lengths) == n_host and as_list(to) == to_host
        assert all(torch.equal(a, b) for a, b in zip(h.images(), want))


def test_free_leaves_bad_lengths_out(cuda_lib):
    """A length below 0 or past what the list holds: no count changes, the sequence is as it was; the others are freed."""
    for bad in (-1, 49, 2 ** 31 - 1):
        h = Held([48, 20, 33], 16, 12, seed=42, width=3, shared=(0,))
        h.d_lengths[0] = bad
        tg.kv_free(h.cache, h.d_uses, h.d_table, h.d_lengths)
        kept = h.lengths[0]
        h.lengths[0] = 0                                         # the definition has nothing to free there
        h.pool.free(h.table, h.lengths)
        torch.cuda.synchronize()
        assert tg.tgemm_last_device_status() == CACHE_ERROR
        assert as_list(h.d_uses) == h.pool.uses and as_list(h.d_lengths) == [bad, 0, 0, 0] and kept == 48


def test_scores_whose_factors_pass_fp32(cuda_lib):
    """The sum times one power of two passes fp32's range, the score itself does not: the best pages all the same."""
    f = Filled(tg, [160], 2, 128, 16, "bf16", seed=43)
    f.k.copy_(torch.where(f.k > 0, 1.0, -1.0) * 2.0 ** 120)      # s = 2^114: a sum of 2^14 and more does not fit beside it
    for i in range(10):
        f.k[int(f.table_host[0, i])] *= 1 + i / 16
    q = (torch.full((1, 4, 128), 2.0 ** -60, device="cuda")).bfloat16()
    to_table, _, _ = select(f, q, 4, 0, 1)
    lists, _ = selection(f, q, 4, 0, 1)
    assert lists[0][0] == [6, 7, 8, 9]
    assert as_list(to_table) == [[[int(f.table_host[0, i]) for i in lists[0][h]] for h in range(2)]]
    # The other way round: a query at the end of the range, its group's others far below, and pages of 0 in between.
    f.k.zero_()
    f.k[int(f.table_host[0, 2])], f.k[int(f.table_host[0, 5])], f.k[int(f.table_host[0, 7])] = 2.0 ** -20, 2.0 ** -21, -2.0 ** -21
    q = torch.full((1, 4, 128), 2.0 ** -70, device="cuda").bfloat16()
    q[0, 1], q[0, 2] = 3e38, -3e38                               # of the two key heads
    to_table, _, _ = select(f, q, 4, 0, 1)
    lists, _ = selection(f, q, 4, 0, 1)
    assert [sorted(x) for x in lists[0]] == [[0, 2, 5, 9], [2, 5, 7, 9]]        # (the least query decides where the largest is against)
    assert as_list(to_table) == [[[int(f.table_host[0, i]) for i in lists[0][h]] for h in range(2)]]


@pytest.mark.parametrize("children,list_pages", [(8, 5), (9, 5), (3, 1024), (3, 1025), (8, 1022), (33, 40), (1, 1400)])
def test_forks_in_one_launch_and_in_two(cuda_lib, children, list_pages):
    """Few children and short lists, and more than a cluster takes: the same pages, counts and rows."""
    h = Held([(list_pages - 1) * 4 - 3, 4 * 4 + 1], 4, list_pages + 100, heads=1, seed=44, width=list_pages)
    parents = [c % 2 for c in range(children)]
    to, to_lengths = torch.full((children, list_pages), -9, dtype=torch.int32, device="cuda"), int32([0] * children)
    want = h.images()
    tg.kv_fork(h.cache, h.d_uses, h.d_table, h.d_lengths, int32(parents), to, to_lengths)
    to_host, n_host = [[-9] * list_pages for _ in range(children)], [0] * children
    for a, z, rows in h.pool.fork(h.table, h.lengths, parents, to_host, n_host):
        for t in want:
            t[z, :rows] = t[a, :rows]
    h.check()
    assert as_list(to) == to_host and as_list(to_lengths) == n_host
    assert all(torch.equal(a, b) for a, b in zip(h.images(), want))
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("sequences,pages", [(8, 160), (8, 161), (9, 160), (1, 160), (30, 1024), (2, 1025)])
def test_compactions_in_one_launch_and_in_two(cuda_lib, sequences, pages):
    h = Held([(pages // 2 // sequences) * 4 - b % 4 for b in range(sequences)], 4, pages, heads=1, seed=45)
    want = h.images()
    to, to_uses, in_use = torch.full_like(h.d_table, -9), torch.full_like(h.d_uses, 77), int32([0])
    tg.kv_compact(h.cache, h.d_uses, h.d_table, h.d_lengths, to, to_uses, in_use)
    moves, n = h.pool.compact(h.table, h.lengths)
    for a, z in moves.items():
        for t in want:
            t[z] = t[a]
    h.check(table=to, uses=to_uses)
    assert as_list(in_use) == [n] and moves
    assert all(torch.equal(a, b) for a, b in zip(h.images(), want))
    assert tg.tgemm_last_device_status() == 0


WIDE_FORKS = [
    # lengths, children, heads, dim, page, cache, layout: rows of all widths, more than a megabyte of last pages, more children
    # than a block has threads
    ([37, 50], 5, 2, 128, 16, "16", "pshd"), ([37, 50], 12, 3, 80, 16, "16", "phsd"), ([20, 31], 4, 1, 256, 24, "16", "pshd"),
    ([37, 90], 6, 2, 256, 16, "e4m3", "phsd"), ([37, 90], 20, 2, 160, 16, "e4m3", "pshd"), ([100, 63, 130], 128, 8, 128, 64, "16", "pshd"),
    ([100, 63, 130], 128, 8, 128, 64, "16", "phsd"), ([300, 200], 30, 8, 256, 128, "e4m3", "pshd"), ([61, 127], 40, 4, 112, 64, "16", "phsd"),
    ([70, 33], 40, 4, 256, 32, "16", "phsd"), ([9, 3, 0, 8], 1200, 1, 64, 4, "16", "pshd"), ([2000], 1030, 2, 96, 8, "16", "phsd"),
]


@pytest.mark.parametrize("case", WIDE_FORKS, ids=lambda c: "-".join(map(str, c[1:])))
def test_fork_of_all_rows(cuda_lib, case):
    lengths, children, heads, dim, page, kind, layout = case
    h = Held(lengths, page, sum(-(-n // page) for n in lengths) + children + 9, heads=heads, dim=dim, kind=kind, layout=layout, seed=50)
    parents = [(7 * c) % (len(lengths) + 1) - 1 for c in range(children)]
    to, to_lengths = torch.full((children, h.width), -9, dtype=torch.int32, device="cuda"), int32([0] * children)
    want = h.images()
    tg.kv_fork(h.cache, h.d_uses, h.d_table, h.d_lengths, int32(parents), to, to_lengths)
    to_host, n_host = [[-9] * h.width for _ in range(children)], [0] * children
    for a, z, rows in h.pool.fork(h.table, h.lengths, parents, to_host, n_host):
        for t in want:
            t[z, :rows] = t[a, :rows]
    h.check()
    assert as_list(to) == to_host and as_list(to_lengths) == n_host
    assert all(torch.equal(a, b) for a, b in zip(h.images(), want))
    tg.kv_free(h.cache, h.d_uses, to, to_lengths)
    h.pool.free(to_host, n_host)
    h.check()
    assert tg.tgemm_last_device_status() == 0


WIDE_COMPACTS = [
    # lengths, heads, dim, page, pages, cache, layout
    ([100, 300], 2, 128, 16, 60, "16", "pshd"), ([100, 300], 3, 80, 16, 60, "16", "phsd"), ([100, 30], 1, 256, 24, 20, "16", "phsd"),
    ([100, 30], 2, 256, 16, 20, "e4m3", "pshd"), ([1000, 700], 8, 128, 64, 60, "16", "phsd"), ([900, 2000], 4, 112, 32, 300, "16", "pshd"),
    ([900, 2000], 4, 256, 32, 300, "e4m3", "phsd"), ([3000] * 10, 2, 128, 16, 3000, "16", "pshd"), ([500] * 70, 1, 64, 64, 700, "16", "pshd"),
    ([3000, 5], 2, 256, 16, 1024, "16", "pshd"),
]


@pytest.mark.parametrize("case", WIDE_COMPACTS, ids=lambda c: f"{len(c[0])}-" + "-".join(map(str, c[1:])))
def test_compaction_of_all_rows(cuda_lib, case):
    lengths, heads, dim, page, pages, kind, layout = case
    h = Held(lengths, page, pages, heads=heads, dim=dim, kind=kind, layout=layout, seed=51)
    bounds = tg.PageBounds(torch.randint(-127, 128, (pages, heads, 2, dim), dtype=torch.int8, generator=h.g).cuda(),
                           torch.rand(pages, heads, generator=h.g).cuda())
    want = h.images() + [bounds.bounds.cpu(), bounds.scale.cpu()]
    to, to_uses, in_use = torch.full_like(h.d_table, -9), torch.full_like(h.d_uses, 77), int32([0])
    tg.kv_compact(h.cache, h.d_uses, h.d_table, h.d_lengths, to, to_uses, in_use, bounds=bounds)
    moves, n = h.pool.compact(h.table, h.lengths)
    for a, z in moves.items():
        for t in want:
            t[z] = t[a]
    h.check(table=to, uses=to_uses)
    assert as_list(in_use) == [n] and moves
    assert all(torch.equal(a, b) for a, b in zip(h.images() + [bounds.bounds.cpu(), bounds.scale.cpu()], want))
    assert tg.tgemm_last_device_status() == 0


@pytest.mark.parametrize("aside", [False, True])
def test_serving_steps_queued(cuda_lib, aside):
    """Steps of all calls, queued one after another with nothing that waits between them; what each has chosen and attended
    to against what was appended until then."""
    heads, group, dim, page, keep, slots, steps, pages = 2, 2, 64, 8, 5, 3, 25, 60
    g = torch.Generator().manual_seed(60)
    cache = tg.PagedCache(*(torch.zeros(pages, page, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    bounds = tg.PageBounds(torch.zeros(pages, heads, 2, dim, dtype=torch.int8, device="cuda"), torch.ones(pages, heads, device="cuda"))
    uses, table = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.zeros(slots, 12, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(slots, dtype=torch.int32, device="cuda")
    rotary = tg.Rotary([100.0 ** (-i / 32) for i in range(32)])
    w = [(1 + 0.1 * torch.randn(dim, generator=g)).bfloat16().cuda() for _ in range(2)]
    prompts = [50, 9, 23]
    starts, counts = int32([0, 50, 59, 82]), int32(prompts)
    positions = int32([i for n in prompts for i in range(n)])

    def rows(n):
        return [(torch.randn(n, m, dim, generator=g) * s).bfloat16().cuda() for m, s in ((heads * group, 2), (heads, 1), (heads, 1))]

    inputs = [rows(sum(prompts))] + [rows(slots) for _ in range(steps)]
    chosen = [torch.zeros(slots, heads, keep, dtype=torch.int32, device="cuda") for _ in range(steps)]
    counted = [torch.zeros(slots, dtype=torch.int32, device="cuda") for _ in range(steps)]
    out = [torch.full((slots, heads * group, dim), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
    ws = tg.attention_decode_workspace(out[0], cache, chosen[0])
    stream = torch.cuda.Stream() if aside else None
    torch.cuda.synchronize()
    for i, (q, k, v) in enumerate(inputs):
        tg.kv_grow(cache, uses, table, lengths, tokens=None if i else counts, stream=stream)
        tg.qk_norm_rope(q, k, lengths if i else positions, rotary, q, k, q_weight=w[0], k_weight=w[1], shift=-1 if i else 0, stream=stream)
        tg.kv_append(cache, k, v, table, lengths, starts=None if i else starts, stream=stream)
        tg.kv_bounds(cache, bounds, table, lengths, starts=None if i else starts, stream=stream)
        if i:
            tg.kv_select(q, cache, bounds, table, lengths, chosen[i - 1], counted[i - 1], first=1, recent=2, stream=stream)
            tg.attention_decode(q, cache, chosen[i - 1], counted[i - 1], out[i - 1], workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert tg.tgemm_last_device_status() == 0
    lists = as_list(table)
    ends = [sum(prompts[:b + 1]) for b in range(slots)]
    kept = [[[t[b] if i else t[ends[b] - prompts[b]:ends[b]] for i, (_, *kv) in enumerate(inputs) for t in [kv[j]]] for j in range(2)]
            for b in range(slots)]
    for i in range(steps):
        q = inputs[i + 1][0]
        for b in range(slots):
            n = prompts[b] + i + 1
            k, v = (torch.cat([kept[b][j][0]] + [x.unsqueeze(0) for x in kept[b][j][1:i + 2]]).double().cpu() for j in range(2))
            assert k.shape[0] == n
            for h in range(heads):
                queries = q[b, h * group:(h + 1) * group].double().cpu()
                scores = [page_score(queries.numpy(), *page_bounds(k[p * page:(p + 1) * page, h].numpy())) if (p + 1) * page <= n else 0.0
                          for p in range(-(-n // page))]
                want = choose(scores, keep, 1, 2)
                assert as_list(chosen[i])[b][h] == [lists[b][p] for p in want] + [-1] * (keep - len(want))
                at = [p * page + s for p in want for s in range(page) if p * page + s < n]
                assert int(counted[i][b]) == len(at)
                p = torch.softmax(k[at, h] @ queries.T * dim ** -0.5, 0)
                o = p.T @ v[at, h]
                # bf16's half step of the output; weights off by 2^-16, their exponents by less than 2^-14
                off = (out[i][b, h * group:(h + 1) * group].double().cpu() - o).abs()
                assert off.max() <= 2.0 ** -8 * o.abs().max() + 2.0 ** -12 * v.abs().max()
