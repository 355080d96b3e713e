"""Attention over an e4m3 cache whose rows are of very different magnitudes, as
kv_append writes them and as a caller may: value = scale * element for every
scale that fp32 holds.

The bound.  A weight times its row's scale, p_j vs_j, is rounded to fp16 under a
reference that puts the largest of the rows met so far (those with an element
that is not 0) at 2^6 or above: relative half a step of fp16, and absolutely at
most 2^-25 of what is 2^6, for each of n rows and elements of at most 448.  The
exponent is t_j plus the scale's, a sum that fp32 rounds to 2^-24 of it, twice
(against the reference).  The rest is as in kv_helpers.attend_bound."""
from __future__ import annotations

import pytest
import torch

from kv_helpers import E4M3, HALF_STEP, TDT, Filled, attend64, score_error, split_e4m3

pytestmark = pytest.mark.gpu


def appended(tg, K, V, page=16, extra_pages=1):
    """One sequence of rows K, V [n, heads, dim] per entry of the lists, written by kv_append into an e4m3 cache."""
    lengths = [len(k) for k in K]
    _, heads, dim = K[0].shape
    width = max(1, max(-(-n // page) for n in lengths))
    pages = len(K) * width + extra_pages
    k, v = (torch.full((pages, page, heads, dim), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = (torch.full((pages, page, heads), float("nan"), device="cuda") for _ in range(2))
    table = torch.randperm(len(K) * width, generator=torch.Generator().manual_seed(pages)).to(torch.int32).view(len(K), width)
    cache = tg.PagedCache(k, v, ks, vs)
    starts = torch.tensor([sum(lengths[:b]) for b in range(len(K) + 1)], dtype=torch.int32)
    out = dict(cache=cache, table=table.cuda(), lengths=torch.tensor(lengths, dtype=torch.int32).cuda(), n=lengths)
    tg.kv_append(cache, torch.cat(K).cuda(), torch.cat(V).cuda(), out["table"], out["lengths"], starts=starts.cuda())
    torch.cuda.synchronize()
    out["k64"], out["v64"], out["vs"] = [], [], []
    for rows, to in ((K, out["k64"]), (V, out["v64"])):
        for x in rows:
            e, s = split_e4m3(x)
            to.append(e.float().double() * s.double().unsqueeze(-1))
            if rows is V:
                out["vs"].append(s.double())
    return out


def check(tg, c, q, dtype, scale):
    """attention_decode with weights against the definition in 64 bits, for every sequence and head."""
    B, H, dim = q.shape
    heads, most = c["cache"].heads, max(c["n"])
    out, w = torch.full_like(q, float("nan"), device="cuda"), torch.zeros(B, heads, most, device="cuda")
    tg.attention_decode(q.cuda(), c["cache"], c["table"], c["lengths"], out, scale=scale, weights=w)
    got, got_w = out.double().cpu(), w.double().cpu()
    for b, n in enumerate(c["n"]):
        o, p, mag, reach, _ = attend64(q[b], c["k64"][b], c["v64"][b], scale)
        vs = c["vs"][b].repeat_interleave(H // heads, 1).T                                  # [H, n]
        some = (c["v64"][b] != 0).any(-1).repeat_interleave(H // heads, 1).T
        exponent = torch.log2(vs[some & (vs > 0)]).abs().max() if (some & (vs > 0)).any() else 0.0
        largest = (p * vs.abs() * some).amax(-1, keepdim=True)
        sums = 2 * (n + 64) * 2.0 ** -24
        e = 2 * score_error(reach, dim, 0.0).unsqueeze(-1) + sums + 4 * 2.0 ** -24 * exponent
        low = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
        bound = (HALF_STEP[dtype] * o.abs() + (1 + HALF_STEP[dtype]) * ((HALF_STEP["fp16"] + 2 * e) * mag + n * 2.0 ** -31 * 448 * largest)
                 + low)
        worst = ((got[b] - o).abs() - bound).max()
        assert ((got[b] - o).abs() <= bound).all(), (b, float(worst), got[b].flatten()[:3], o.flatten()[:3])
        add = p.view(heads, H // heads, n).sum(1)
        ew = (2 * score_error(reach, dim, 0.0) + sums).view(heads, -1).amax(-1, keepdim=True)
        assert ((got_w[b, :, :n] - add).abs() <= (2.0 ** -22 + 2 * ew) * add).all(), b
    assert tg.tgemm_last_device_status() == 0


def rows(n, heads, dim, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, dim, generator=g, dtype=torch.float64) * size).to(TDT[dtype])


@pytest.mark.parametrize("size", [2.0 ** -126, 1e-36, 1e-30, 1e-20, 1e-7, 1e10, 1e30])
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 12), (256, 8)])
def test_values_of_every_magnitude(cuda_lib, dim, group, size):
    n = [700, 1, 40]
    K, V = [rows(i, 2, dim, "bf16", i) for i in n], [rows(i, 2, dim, "bf16", i + 1, size) for i in n]
    q = rows(3, 2 * group, dim, "bf16", 5)
    check(cuda_lib, appended(cuda_lib, K, V), q, "bf16", dim ** -0.5)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_of_many_magnitudes_in_one_sequence(cuda_lib, dtype):
    """Rows over the type's range, the small ones in dims where the large ones are 0."""
    g = torch.Generator().manual_seed(2)
    K, V = rows(900, 2, 64, dtype, 3), rows(900, 2, 64, dtype, 4).double()
    lo, hi = (-12, 8) if dtype == "fp16" else (-16, 100)
    size = torch.randint(lo, hi, (900, 2, 1), generator=g).double()
    V = V * torch.exp2(size)
    V[..., :32] *= (size < (lo + hi) / 2)
    V[..., 32:] *= (size >= (lo + hi) / 2)
    check(cuda_lib, appended(cuda_lib, [K], [V.to(TDT[dtype])]), rows(1, 8, 64, dtype, 6), dtype, 0.125)


@pytest.mark.parametrize("apart", [60, 110, 126])
def test_a_large_scale_on_a_light_row(cuda_lib, apart):
    """The row that carries almost all weight has a scale 2^apart below the others': the weights stay those of the scores."""
    n, dim = 500, 64
    K, V = torch.zeros(n, 1, dim).bfloat16(), rows(n, 1, dim, "bf16", 7, 2.0 ** (apart - 63))
    K[100] = 1.0
    V[100] = rows(1, 1, dim, "bf16", 8, 2.0 ** -63)[0]
    check(cuda_lib, appended(cuda_lib, [K], [V]), torch.ones(1, 2, dim).bfloat16(), "bf16", 20 * 0.6931 / dim)


@pytest.mark.parametrize("value", [0.0, 2.0 ** -149, 2.0 ** -127, 2.0 ** -101])
def test_scales_that_are_nothing_or_nearly(cuda_lib, value):
    """A scale of 0 makes its row 0 whatever its elements are; one below fp32's normal range counts as what it is."""
    tg = cuda_lib
    f = Filled(tg, [300, 20], 2, 64, 16, "bf16", "e4m3", seed=3)
    c = dict(cache=f.cache, table=f.table, lengths=f.lengths, n=[300, 20], k64=f.k64)
    f.vs.nan_to_num_(0.0)
    f.vs.fill_(value)
    c["v64"], c["vs"] = [], []
    for b, n in enumerate(c["n"]):
        pos = torch.arange(n)
        elements = f.v.view(torch.uint8)[f.table_host[b].long()[pos // 16].cuda(), (pos % 16).cuda()].view(E4M3).double().cpu()
        c["v64"].append(elements * value)
        c["vs"].append(torch.full((n, 2), value, dtype=torch.float64))
    check(tg, c, rows(2, 4, 64, "bf16", 4), "bf16", 0.125)


@pytest.mark.parametrize("dtype,value", [("bf16", 1.0), ("bf16", 1e-3), ("bf16", 1e-6), ("bf16", 1e-7), ("bf16", 1e-30), ("fp16", 1.0),
                                         ("fp16", 2e-4)])
@pytest.mark.parametrize("ahead", [0.0, 14.4, 26.0, 60.0])
@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_one_row_of_zeros_beside_small_values(cuda_lib, zero, ahead, dtype, value):
    """A row of zeros, 2^ahead times as heavy as each other row, adds nothing and costs the others no precision: one
    key head that the whole GPU shares, and many that one block each takes."""
    dim = 64
    for batch, n, heads in ((1, 600, 1), (1, 9000, 1), (8, 300, 38), (2, 2, 1)):
        K, V = [], []
        for b in range(batch):
            k, v = torch.zeros(n, heads, dim), rows(n, heads, dim, dtype, b + n, 1.0).float().abs().clamp(0.25, 2.0) * value
            at = (n // 3) * (b % 3)
            k[at] = 1.0
            v[at] = zero
            K.append(k.to(TDT[dtype]))
            V.append(v.to(TDT[dtype]))
        c = appended(cuda_lib, K, V)
        assert (torch.cat(c["vs"]) == 1).any()
        check(cuda_lib, c, torch.ones(batch, heads * 2, dim, dtype=TDT[dtype]), dtype, ahead * 0.6931471805599453 / dim)


@pytest.mark.parametrize("dim,group", [(64, 3), (80, 16), (128, 8), (256, 4)])
def test_rows_of_zeros_everywhere(cuda_lib, dim, group):
    """Every third row zero, and a sequence of nothing else."""
    n = [900, 50, 1]
    K, V = [rows(i, 2, dim, "bf16", i, 3.0) for i in n], [rows(i, 2, dim, "bf16", i + 1, 1e-4) for i in n]
    V[0][::3] = 0
    V[1][:] = 0
    c = appended(cuda_lib, K, V)
    check(cuda_lib, c, rows(3, 2 * group, dim, "bf16", 5, 3.0), "bf16", dim ** -0.5)
