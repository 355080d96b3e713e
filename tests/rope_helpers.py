"""Head norms with the position rotation in 64 bits, and the bounds of what fp32 may be off by."""
from __future__ import annotations

import torch

TDT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
SMALLEST = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}      # half the least subnormal


def members(pairs, interleaved):
    """The elements of each pair."""
    i = torch.arange(pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)


def angles64(positions, frequencies, axes, shift=0):
    """[tokens, 1, pairs]"""
    f = torch.tensor(frequencies, dtype=torch.float64)
    return ((positions.cpu().double() + shift)[torch.tensor(axes, dtype=torch.long)].T * f).unsqueeze(1)


def turn64(x, angle, interleaved):
    a, b = members(angle.shape[-1], interleaved)
    y = x.clone()
    c, s = torch.cos(angle), torch.sin(angle)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def reach(x, pairs, interleaved):
    """|a| + |b| of an element's pair, |x| of those that do not turn."""
    a, b = members(pairs, interleaved)
    m = x.abs()
    s = m[..., a] + m[..., b]
    m[..., a], m[..., b] = s, s
    return m


def forward64(x, w, eps, angle, interleaved):
    """(y, what bounds its fp32 error before the rounding)"""
    x = x.double().cpu()
    dim = x.shape[-1]
    v = x if eps is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    v = v if w is None else v * w.double().cpu()
    # r: the sum's dim roundings, halved by the root, and the root's own; three products; an angle off by 2^-22 at most
    # (fp32's half step of half a turn), its sine and cosine by 2^-22.
    e = (dim / 2 + 16) * 2.0 ** -24 + 2.0 ** -21
    return turn64(v, angle, interleaved), e * reach(v, angle.shape[-1], interleaved)


def backward64(x, w, dy, eps, angle, interleaved):
    """(dx, its error's bound, dw, its error's bound)"""
    x, dy = x.double().cpu(), dy.double().cpu()
    dim = x.shape[-1]
    g = turn64(dy, -angle, interleaved)
    mg = reach(dy, angle.shape[-1], interleaved)
    e_g = 8 * 2.0 ** -24 + 2.0 ** -21
    if eps is None:
        return g, e_g * mg, None, None
    w = torch.ones(dim, dtype=torch.float64) if w is None else w.double().cpu()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dot = (g * w * x).sum(-1, keepdim=True)
    dx = r * (g * w - x * r * r * dot / dim)
    e = (dim / 2 + 16) * 2.0 ** -24
    size = (mg * w.abs() * x.abs()).sum(-1, keepdim=True)
    bound = r * w.abs() * mg * (e_g + 2 * e) + x.abs() * r ** 3 * size / dim * (e_g + 6 * e)
    n = x.shape[0] * x.shape[1]
    dw = (g * x * r).sum((0, 1))
    return dx, bound, dw, (mg * x.abs() * r).sum((0, 1)) * (e_g + e + (n + 64) * 2.0 ** -24)


def close(got, want, bound, dtype):
    """got is want rounded once, but for `bound`."""
    u = HALF_STEP[dtype]
    off = (got.double().cpu() - want).abs()
    room = u * want.abs() + (1 + u) * bound + SMALLEST[dtype]
    assert got.isfinite().all()
    bad = off > room
    assert not bad.any(), (off - room).max().item()
