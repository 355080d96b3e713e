"""Shared helpers of the paged-cache tests: caches in several layouts whose
unused rows hold NaN, and the operators' definitions in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

TDT = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
BAD_PAGE = 0x7FFFFFFF


def make_pool(pages, page, heads, dim, dtype, layout, device):
    """k and v pools [pages, page, heads, dim] filled with NaN, as views of the given memory layout."""
    if layout == "pshd":
        k, v = (torch.empty(pages, page, heads, dim, dtype=dtype, device=device) for _ in range(2))
    elif layout == "phsd":          # a page's rows of one head together
        k, v = (torch.empty(pages, heads, page, dim, dtype=dtype, device=device).transpose(1, 2) for _ in range(2))
    elif layout == "both":          # one pool that holds keys and values side by side, with padded rows
        both = torch.empty(pages, 2, page, heads, dim + 16, dtype=dtype, device=device)
        k, v = both[:, 0, :, :, :dim], both[:, 1, :, :, :dim]
    else:
        raise ValueError(layout)
    for t in (k, v):
        if dtype == E4M3:
            t.view(torch.uint8).fill_(0x7F)
        else:
            t.fill_(float("nan"))
    return k, v


def make_table(lengths, page, extra, seed, width=None, past=BAD_PAGE):
    """A shuffled page table; entries past a sequence's own pages hold `past`."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + extra
    order = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    table = np.full((len(lengths), width or max([1] + need)), past, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table), pages


def split_e4m3(x):
    """Elements and scales of rows x [..., dim] by the definition: max |x| / 448, x / scale rounded."""
    x = x.float()
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return (x / scale.unsqueeze(-1)).to(E4M3), scale


class Filled:
    """A cache on the GPU that holds random rows for sequences of the given
    lengths, and those rows in 64 bits per sequence: k64[b], v64[b] [n, heads, dim]."""

    def __init__(self, tg, lengths, heads, dim, page, dtype, cache="16", layout="pshd", seed=0, k_gain=1.0, width=None,
                 extra=2):
        g = torch.Generator().manual_seed(seed)
        self.table_host, pages = make_table(lengths, page, extra, seed, width)
        ctype = E4M3 if cache == "e4m3" else TDT[dtype]
        self.k, self.v = make_pool(pages, page, heads, dim, ctype, layout, "cuda")
        self.ks = self.vs = None
        if cache == "e4m3":
            self.ks, self.vs = (torch.full((pages, page, heads), float("nan"), device="cuda") for _ in range(2))
        self.k64, self.v64 = [], []
        for b, n in enumerate(lengths):
            pos = torch.arange(n)
            pg, slot = self.table_host[b].long()[pos // page].cuda(), (pos % page).cuda()
            for pool, sc, keep, gain in ((self.k, self.ks, self.k64, k_gain), (self.v, self.vs, self.v64, 1.0)):
                x = (torch.randn(n, heads, dim, generator=g) * gain).to(TDT[dtype])
                if cache == "e4m3":
                    e, s = split_e4m3(x)
                    flat = pool.view(torch.uint8)
                    flat[pg, slot] = e.view(torch.uint8).cuda()
                    sc[pg, slot] = s.cuda()
                    keep.append(e.float().double() * s.double().unsqueeze(-1))
                else:
                    pool[pg, slot] = x.cuda()
                    keep.append(x.double())
        self.lengths_host = list(lengths)
        self.table = self.table_host.cuda()
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.cache = tg.PagedCache(self.k, self.v, self.ks, self.vs)
        self.heads, self.dim, self.page, self.dtype, self.kind = heads, dim, page, dtype, cache


def attend64(q, k, v, scale, cap=0.0, keep=None):
    """One sequence in 64 bits: q [q_heads, dim], k, v [n, heads, dim]; keep: the positions that count.
    Returns o, p [q_heads, n], and per query head the bounds' ingredients: sum p |v|, the largest
    sum |q k| * |scale|, the largest |v|."""
    H, D = q.shape
    n, heads, _ = k.shape
    group = H // heads
    o, mag = torch.zeros(H, D, dtype=torch.float64), torch.zeros(H, D, dtype=torch.float64)
    p_all, reach = torch.zeros(H, n, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
    idx = torch.arange(n) if keep is None else keep
    if idx.numel() == 0:
        return o, p_all, mag, reach, torch.zeros(H, dtype=torch.float64)
    top = torch.zeros(H, dtype=torch.float64)
    for h in range(H):
        kk, vv, qq = k[idx, h // group], v[idx, h // group], q[h].double()
        s = (kk @ qq) * scale
        if cap > 0:
            s = cap * torch.tanh(s / cap)
        e = torch.exp(s - s.max())
        p = e / e.sum()
        o[h], mag[h] = p @ vv, p @ vv.abs()
        p_all[h, idx] = p
        reach[h] = (kk.abs() @ qq.abs()).max() * abs(scale)
        top[h] = vv.abs().max()
    return o, p_all, mag, reach, top


def score_error(reach, dim, cap):
    """Bound of the error of a softmax weight's exponent: the dot product's dim
    roundings in fp32 (doubled for the tensor core's internal alignment), a few
    more for the scale and the change of base, and, capped, the tanh's absolute
    error of a few units of 2^-24 times the cap (its slope is at most 1)."""
    return 2 * (dim + 8) * 2.0 ** -24 * reach + 16 * 2.0 ** -24 * cap + 2.0 ** -22


def attend_bound(o, mag, reach, top, n, dim, dtype, p_dtype, cap):
    """|out - o| allowed: the output's rounding; every weight's relative error
    (exponent, its rounding to p_dtype before the second product, and the fp32
    sums over n positions) against sum p |v|, once for the products and once for
    the divisor; fp16 weights below 2^-14 are off by up to 2^-25 absolutely."""
    e = 2 * score_error(reach, dim, cap).unsqueeze(-1) + 2 * (n + 64) * 2.0 ** -24
    u_p = HALF_STEP[p_dtype]
    small = n * 2.0 ** -25 * top.unsqueeze(-1) if p_dtype == "fp16" else 0.0
    low = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
    return HALF_STEP[dtype] * o.abs() + (1 + HALF_STEP[dtype]) * ((u_p + 2 * e) * mag + small) + low


def evict_reference(weights, n, keep, recent):
    """Positions kept of one head's weights (float32 numpy [>= n]), ascending."""
    k = min(n, keep)
    r = min(recent, k)
    w = [(-np.inf, 0) if np.isnan(x) else (float(x), 1) for x in weights[:n - r]]
    order = sorted(range(n - r), key=lambda j: (-w[j][1], -w[j][0] if w[j][1] else 0.0, j))
    return sorted(order[:k - r]) + list(range(n - r, n))
