"""The paged key-value cache: writing new tokens, attention of one new token
per sequence, and eviction by accumulated attention weight.

The computation lives in the CUDA library (csrc/kv_*.cuh, C ABI in
include/tgemm.h); this module checks and marshals torch tensors.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b

_DT = {torch.float16: _b.TGEMM_F16, torch.bfloat16: _b.TGEMM_BF16}
_E4M3 = torch.float8_e4m3fn


class PagedCache:
    """Keys and values in pages.

    k and v are the pools, [pages, page_size, heads, dim] in float16, bfloat16
    or float8_e4m3fn, with equal strides (any layout: a transposed view of a
    [pages, heads, page_size, dim] tensor, or two views of one pool).  An e4m3
    cache also has k_scale and v_scale, float32 [pages, page_size, heads], one
    factor per row (value = scale * element).  The object keeps the tensors and
    their description for the calls below; it owns nothing else.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor = None, v_scale: torch.Tensor = None):
        for name, t in (("k", k), ("v", v)):
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{name} must be [pages, page_size, heads, dim] with unit stride of dim")
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must share shape, strides, dtype and device")
        if k.dtype not in _DT and k.dtype != _E4M3:
            raise ValueError("k and v must be float16, bfloat16 or float8_e4m3fn")
        e4m3 = k.dtype == _E4M3
        if e4m3:
            if k_scale is None or v_scale is None:
                raise ValueError("an e4m3 cache needs k_scale and v_scale")
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t.dtype != torch.float32 or t.shape != k.shape[:3] or t.device != k.device:
                    raise ValueError(f"{name} must be float32 [pages, page_size, heads] on the pools' device")
            if k_scale.stride() != v_scale.stride():
                raise ValueError("k_scale and v_scale must share strides")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("only an e4m3 cache has scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.page_size, self.heads, self.dim = k.shape
        self.dtype, self.device, self.e4m3 = k.dtype, k.device, e4m3
        c = _b.KvCache()
        c.k, c.v = k.data_ptr() or None, v.data_ptr() or None
        c.pages, c.page_size, c.heads, c.dim, c.e4m3 = self.pages, self.page_size, self.heads, self.dim, int(e4m3)
        c.page_stride, c.slot_stride, c.head_stride = k.stride()[:3]
        if e4m3:
            c.k_scale, c.v_scale = k_scale.data_ptr() or None, v_scale.data_ptr() or None
            c.scale_page_stride, c.scale_slot_stride, c.scale_head_stride = k_scale.stride()
        self._struct = c
        self._ref = ctypes.byref(c)


def _table(page_table, lengths, cache, need_lengths=True):
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("the page table must be int32 [batch, pages] with unit stride of pages")
    batch, width = page_table.shape
    if page_table.device != cache.device:
        raise ValueError("the page table must be on the cache's device")
    if need_lengths:
        _vector("lengths", lengths, batch, cache)
    return batch, width, page_table.stride(0)


def _vector(name, t, n, cache):
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1) or t.device != cache.device:
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on the cache's device")


def _weights(name, w, batch, cache):
    """(pointer, width, batch stride, head stride) of accumulated weights, or zeros for None."""
    if w is None:
        return 0, 0, 0, 0
    if w.dim() != 3 or w.dtype != torch.float32 or w.device != cache.device or tuple(w.shape[:2]) != (batch, cache.heads) or (
            w.shape[2] > 1 and w.stride(2) != 1):
        raise ValueError(f"{name} must be float32 [batch, heads, positions] on the cache's device with unit stride of positions")
    return w.data_ptr(), w.shape[2], w.stride(0), w.stride(1)


def _launch(cache, stream, where, call):
    """call(stream handle) with the cache's device current; raises on a status."""
    dev = cache.device
    if dev.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    if dev.index == torch.cuda.current_device():
        st = call(s.cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = call(s.cuda_stream)
    if st != 0:
        raise _b.TgemmError(st, where)


def _call_dtype(name, t, cache):
    code = _DT.get(t.dtype)
    if code is None or (not cache.e4m3 and t.dtype != cache.dtype):
        raise ValueError(f"{name} must be float16 or bfloat16, and the cache's dtype unless that is e4m3")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on the cache's device")
    return code


def kv_append(cache: PagedCache, K: torch.Tensor, V: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
              starts: torch.Tensor = None, weights: torch.Tensor = None, stream=None) -> None:
    """Write the newest tokens' keys and values, [tokens, heads, dim], into the
    cache.  Sequence b brings tokens starts[b] .. starts[b + 1] - 1 (starts:
    int32 [batch + 1]; None: one token each), which lengths[b] counts already:
    its last token goes to position lengths[b] - 1.  weights (float32 [batch,
    heads, positions]) are set to zero there."""
    batch, width, stride = _table(page_table, lengths, cache)
    if K.dim() != 3 or K.shape != V.shape or tuple(K.shape[1:]) != (cache.heads, cache.dim):
        raise ValueError("K and V must be [tokens, heads, dim] of the cache's heads and dim")
    sk = K.stride()
    if sk != V.stride() or sk[2] != 1:
        raise ValueError("K and V must share strides, with unit stride of dim")
    if K.dtype != V.dtype or K.device != V.device:
        raise ValueError("K and V must share dtype and device")
    code = _call_dtype("K", K, cache)
    if starts is not None:
        _vector("starts", starts, batch + 1, cache)
    elif K.shape[0] != batch:
        raise ValueError("without starts every sequence brings one token")
    w = _weights("weights", weights, batch, cache)
    args = (cache._ref, K.data_ptr(), V.data_ptr(), K.shape[0], sk[0], sk[1],
            starts.data_ptr() if starts is not None else 0, page_table.data_ptr(), width, stride, lengths.data_ptr(),
            batch, *w, code)
    _launch(cache, stream, "tgemm_kv_append", lambda s: _b.tgemm_kv_append(*args, s))


def attention_decode_workspace(Q: torch.Tensor, cache: PagedCache, page_table: torch.Tensor,
                               weights: bool = False) -> torch.Tensor:
    """A workspace for attention_decode() with operands of these shapes (or
    smaller ones): zeroed device memory, to be kept between calls.  Calls that
    may overlap on the GPU need one each."""
    n = _b.tgemm_attention_decode_workspace(Q.shape[0], Q.shape[1], cache.heads, cache.dim,
                                            page_table.shape[1] * cache.page_size, bool(weights))
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def attention_decode(Q: torch.Tensor, cache: PagedCache, page_table: torch.Tensor, lengths: torch.Tensor,
                     O: torch.Tensor, scale: float = None, cap: float = 0.0, window: int = 0,
                     weights: torch.Tensor = None, workspace: torch.Tensor = None, stream=None) -> torch.Tensor:
    """O[b, h] = attention of the new token's query Q[b, h] over the first
    lengths[b] positions of sequence b's cache (the last `window` of them, if
    that is not 0); Q and O are [batch, q_heads, dim], q_heads a multiple of the
    cache's heads.  scale defaults to 1 / sqrt(dim); cap > 0 passes the scaled
    scores through cap * tanh(s / cap).  weights (float32 [batch, heads,
    positions]) grow by each group's summed attention.  Without a workspace one
    is allocated and zeroed for the call."""
    batch, width, stride = _table(page_table, lengths, cache)
    if Q.dim() != 3 or Q.shape != O.shape or Q.shape[0] != batch or Q.shape[2] != cache.dim or Q.shape[1] % cache.heads:
        raise ValueError("Q and O must be [batch, q_heads, dim], q_heads a multiple of the cache's heads")
    sq, so = Q.stride(), O.stride()
    if sq[2] != 1 or so[2] != 1:
        raise ValueError("Q and O need unit stride of dim")
    if O.dtype != Q.dtype or O.device != Q.device:
        raise ValueError("Q and O must share dtype and device")
    code = _call_dtype("Q", Q, cache)
    if scale is None:
        scale = cache.dim ** -0.5
    w = _weights("weights", weights, batch, cache)
    if workspace is None:
        with torch.cuda.stream(stream):   # the zeros belong to the stream that uses them
            workspace = attention_decode_workspace(Q, cache, page_table, weights is not None)
    elif workspace.device != cache.device or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the cache's device")
    args = (cache._ref, Q.data_ptr(), O.data_ptr(), batch, Q.shape[1], sq[0], sq[1], so[0], so[1],
            page_table.data_ptr(), width, stride, lengths.data_ptr(), scale, cap, window, *w, workspace.data_ptr(),
            workspace.nbytes, code)
    _launch(cache, stream, "tgemm_attention_decode", lambda s: _b.tgemm_attention_decode(*args, s))
    return O


def kv_evict(cache: PagedCache, page_table: torch.Tensor, lengths: torch.Tensor, weights: torch.Tensor,
             to_cache: PagedCache, to_page_table: torch.Tensor, kept: torch.Tensor, to_lengths: torch.Tensor,
             to_weights: torch.Tensor, recent: int = 0, stream=None) -> None:
    """Bring every sequence back to at most keep = kept.shape[2] positions: each
    head keeps the last `recent` and, of those before, the ones of largest
    weight (ties to the lowest position).  Their rows are copied in order to the
    pages of to_page_table in to_cache (which may describe the same pools; the
    pages written must not be among those read).  Written besides: kept (int32
    [batch, heads, keep], -1 where a sequence has fewer), to_lengths (int32
    [batch]) and to_weights (float32 [batch, heads, at least keep])."""
    batch, width, stride = _table(page_table, lengths, cache)
    to_batch, to_width, to_stride = _table(to_page_table, None, to_cache, need_lengths=False)
    if to_batch != batch or to_cache.device != cache.device or (to_cache.dtype, to_cache.heads, to_cache.dim) != (
            cache.dtype, cache.heads, cache.dim):
        raise ValueError("both caches must share dtype, heads, dim and device, both page tables the batch")
    if kept.dim() != 3 or kept.dtype != torch.int32 or not kept.is_contiguous() or kept.device != cache.device or tuple(
            kept.shape[:2]) != (batch, cache.heads):
        raise ValueError("kept must be a contiguous int32 [batch, heads, keep] tensor on the cache's device")
    _vector("to_lengths", to_lengths, batch, cache)
    keep = kept.shape[2]
    if to_weights.dim() != 3 or to_weights.shape[2] < keep:
        raise ValueError("to_weights must hold at least keep positions")
    args = (cache._ref, page_table.data_ptr(), width, stride, lengths.data_ptr(), batch,
            *_weights("weights", weights, batch, cache), to_cache._ref, to_page_table.data_ptr(), to_width, to_stride,
            keep, recent, kept.data_ptr(), to_lengths.data_ptr(), *_weights("to_weights", to_weights, batch, cache))
    _launch(cache, stream, "tgemm_kv_evict", lambda s: _b.tgemm_kv_evict(*args, s))
