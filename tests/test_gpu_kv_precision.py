"""How exactly attention over the paged cache keeps its softmax weights: as
fp32 values split into two of 16 bits, so that an output that comes of large
values of both signs is as good as its weights.

The bound.  Besides its exponent (kv_helpers.score_error) and the fp32 sums, a
weight is off by 2^-16 of itself (bf16 products) or 2^-21 (fp16; e4m3 rows are
widened to it), or by 2^-25 of what is 2^6 or more."""
from __future__ import annotations

import pytest
import torch

from kv_helpers import HALF_STEP, TDT, Filled, attend64, score_error

pytestmark = pytest.mark.gpu

SPLIT = {"fp16": 2.0 ** -21, "bf16": 2.0 ** -16}
KINDS = [("16", "fp16"), ("16", "bf16"), ("e4m3", "fp16"), ("e4m3", "bf16")]


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("dim,group,width", [(64, 1, None), (64, 12, None), (64, 16, 4000), (64, 24, 4000), (80, 3, None), (128, 8, None),
                                             (128, 16, 4000), (128, 24, 4000), (256, 5, None)])
def test_outputs_that_cancel(cuda_lib, dim, group, width, cache, dtype):
    """Values of the same size and either sign: the weights' own errors are what is left.  Few positions, so that
    these do not average out."""
    lengths = [2, 3, 5, 17, 40]
    f = Filled(cuda_lib, lengths, 4, dim, 16, dtype, cache, seed=dim + group, width=width)
    if cache == "e4m3":
        f.vs.nan_to_num_(1.0)
        f.vs.fill_(1.0)
    for b, n in enumerate(lengths):
        for j in range(n):
            page, sign = int(f.table_host[b, j // 16]), 1.0 - 2.0 * (j % 2)
            if cache == "e4m3":
                f.v.view(torch.uint8)[page, j % 16] = 0x38 if sign > 0 else 0xB8
            else:
                f.v[page, j % 16] = sign
            f.v64[b][j] = sign
    q = (torch.randn(len(lengths), 4 * group, dim, generator=torch.Generator().manual_seed(1)) * 0.1).to(TDT[dtype])
    out = torch.empty_like(q, device="cuda")
    cuda_lib.attention_decode(q.cuda(), f.cache, f.table, f.lengths, out, scale=dim ** -0.5)
    for b, n in enumerate(lengths):
        o, p, mag, reach, top = attend64(q[b], f.k64[b], f.v64[b], dim ** -0.5)
        e = 2 * score_error(reach, dim, 0.0).unsqueeze(-1) + 2 * (n + 64) * 2.0 ** -24
        u = SPLIT["fp16" if cache == "e4m3" else dtype]
        low = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
        bound = HALF_STEP[dtype] * o.abs() + (1 + HALF_STEP[dtype]) * ((u + 2 * e) * mag + n * 2.0 ** -31 * top.unsqueeze(-1)) + low
        worst = ((out[b].double().cpu() - o).abs() - bound).max()
        assert worst <= 0, (b, float(worst))
    assert cuda_lib.tgemm_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,group,width", [(64, 1, None), (64, 16, 4000), (128, 8, None), (128, 24, 4000), (256, 3, None)])
def test_an_infinite_value_stays_infinite(cuda_lib, dim, group, width, dtype):
    """An infinity in a row that counts makes its head's outputs in that dim infinite, with its sign, and no other:
    on the heaviest row (whose weight is a power of two) as on others."""
    f = Filled(cuda_lib, [1, 60, 300], 2, dim, 16, dtype, seed=dim, width=width)
    where = [(0, 0, 0, 3, 1.0), (1, 17, 1, 5, -1.0), (2, 0, 0, 8, 1.0), (2, 299, 1, 0, -1.0), (2, 100, 0, 9, -1.0)]
    for b, j, h, d, sign in where:
        f.v[int(f.table_host[b, j // 16]), j % 16, h, d] = sign * float("inf")
    q = (torch.randn(3, 2 * group, dim, generator=torch.Generator().manual_seed(2)) * 0.5).to(TDT[dtype]).cuda()
    for weigh in (q, torch.zeros_like(q)):          # scores as they come, and all equal: every weight a power of two
        out = torch.empty_like(q)
        cuda_lib.attention_decode(weigh, f.cache, f.table, f.lengths, out)
        want = torch.zeros(3, 2 * group, dim)
        for b, j, h, d, sign in where:
            want[b, h * group:(h + 1) * group, d] = sign
        got = out.float().cpu()
        assert not torch.isnan(got).any()
        assert torch.equal(torch.isinf(got), want != 0)
        assert (torch.sign(got)[want != 0] == want[want != 0]).all()


@pytest.mark.parametrize("cache,dtype", KINDS)
@pytest.mark.parametrize("low,high", [(0.150, 0.176), (0.30, 0.33), (0.01, 0.04), (0.80, 0.84)])
def test_capped_scores_are_as_good_as_others(cuda_lib, low, high, cache, dtype):
    """Two positions whose q k is exact: the added weight of the lighter one shows the error of their scores'
    difference.  Of each score, in units of 2^-24 of it: the quotient's product with q k 1, tanh 2, the product with
    the cap 1 (the quotient scale / cap and the cap are the same for both: 3 of the difference, with the subtraction
    of the reference); then 2^-22 for each of two exponentials and the join's factor, and a few roundings of the sum
    and the quotient."""
    dim, heads, cap = 64, 8, 1000.0
    f = Filled(cuda_lib, [2], heads, dim, 16, dtype, cache, seed=1)
    page = int(f.table_host[0, 0])
    k = torch.tensor([[round(low * 256) / 256 * 512 + h, round(high * 256) / 256 * 512 + 2 * h] for h in range(heads)],
                     dtype=torch.float64)                                   # [heads, 2], whole numbers below 512
    for pool in (f.k, f.v):
        pool.view(torch.uint8)[page, :2] = 0
    if cache == "e4m3":         # an element of 1, the rest in the row's scale
        f.vs[page, :2] = 1.0
        f.ks[page, :2] = k.T.float().cuda()
        f.k.view(torch.uint8)[page, :2, :, 0] = 0x38
    else:
        f.k[page, :2, :, 0] = (k.T / 2).to(TDT[dtype]).cuda() * 2
        k = f.k[page, :2, :, 0].double().cpu().T
    q = torch.zeros(1, heads, dim, dtype=TDT[dtype])
    q[0, :, 0] = 1.0
    out, w = torch.empty_like(q, device="cuda"), torch.zeros(1, heads, 2, device="cuda")
    for i in range(64):
        scale = 2.0 * (1 - i / 5000)
        w.zero_()
        cuda_lib.attention_decode(q.cuda(), f.cache, f.table, f.lengths, out, scale=scale, cap=cap, weights=w)
        s = cap * torch.tanh(k * scale / cap)
        p = torch.softmax(s, 1)
        e = 2.0 ** -24 * (4 * s.abs().sum(1) + 3 * (s[:, 1] - s[:, 0]).abs() + 16) + 3 * 2.0 ** -22
        assert ((w[0, :, 0].double().cpu() - p[:, 0]).abs() <= e * p[:, 0]).all(), i
    assert cuda_lib.tgemm_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("cap", [1e-10, 1e-30, 1e-45, 1e-300])
def test_caps_near_zero_over_keys_of_zero(cuda_lib, cap, dtype):
    """e4m3: scores that all become 0, of keys with scales above 1, some with elements of 0: the average of the
    values."""
    f = Filled(cuda_lib, [100], 2, 64, 16, dtype, "e4m3", seed=8)
    f.ks.nan_to_num_(1.0)
    f.ks.fill_(37.0)
    f.k.view(torch.uint8)[f.table_host[0, 2].item()] = 0
    q = (torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(3)) * 5000).to(TDT[dtype])
    q[0, 3] = 0
    out = torch.full_like(q, float("nan"), device="cuda")
    cuda_lib.attention_decode(q.cuda(), f.cache, f.table, f.lengths, out, cap=cap)
    o, p, mag, reach, top = attend64(q[0], torch.zeros_like(f.k64[0]), f.v64[0], 0.0)
    e = 2 * 2.0 ** -22 + 2 * (100 + 64) * 2.0 ** -24 + 4 * cap
    bound = (HALF_STEP[dtype] * o.abs() + (1 + HALF_STEP[dtype]) * ((SPLIT["fp16"] + 2 * e) * mag + 100 * 2.0 ** -31 * top.unsqueeze(-1))
             + (2.0 ** -25 if dtype == "fp16" else 2.0 ** -134))
    assert ((out[0].double().cpu() - o).abs() <= bound).all()
