"""The paged key-value cache: writing new tokens, attention of one new token
per sequence, and eviction by accumulated attention weight.

The computation lives in the CUDA library (csrc/kv_*.cuh, C ABI in
include/tgemm.h); this module checks torch tensors and packs their addresses
and sizes into the calls' argument structures.  A call costs the host a few
microseconds, so every tensor attribute is read once and by its cheapest name
(get_device() rather than device).
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b

_F16, _BF16, _E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
_DT = {_F16: _b.TGEMM_F16, _BF16: _b.TGEMM_BF16}
_NO_WEIGHTS = (0, 0, 0, 0)
# The current stream's handle and the current device, without building the
# objects that torch.cuda's functions return (about a microsecond a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_append, _decode, _evict = _b.KV_APPEND_ARGS.pack, _b.ATTENTION_DECODE_ARGS.pack, _b.KV_EVICT_ARGS.pack


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
        self._address = ctypes.addressof(c)
        self._index = k.get_device()          # -1: not on a GPU
        self._dtypes = (_F16, _BF16) if e4m3 else (k.dtype,)


def _table(page_table, index):
    """(pages, width, stride, batch) of a page table."""
    shape, stride = page_table.shape, page_table.stride()
    if len(shape) != 2 or page_table.dtype is not torch.int32 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError("the page table must be int32 [batch, pages] with unit stride of pages")
    if page_table.get_device() != index:
        raise ValueError("the page table must be on the cache's device")
    return page_table.data_ptr(), shape[1], stride[0], shape[0]


def _vector(name, t, n, index):
    """The address of a contiguous int32 [n] tensor."""
    if t.dtype is not torch.int32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on the cache's device")
    return t.data_ptr()


def _weights(name, w, batch, heads, index):
    """(address, width, batch stride, head stride) of accumulated weights."""
    shape, stride = w.shape, w.stride()
    if (len(shape) != 3 or w.dtype is not torch.float32 or shape[0] != batch or shape[1] != heads
            or (stride[2] != 1 and shape[2] > 1) or w.get_device() != index):
        raise ValueError(f"{name} must be float32 [batch, heads, positions] on the cache's device with unit stride of positions")
    return w.data_ptr(), shape[2], stride[0], stride[1]


def _launch(index, stream, fn, args):
    """fn(args, stream) with the cache's device current; raises on a status."""
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _current_device():
        st = fn(args, s)
    else:
        with torch.cuda.device(index):
            st = fn(args, s)
    if st != 0:
        raise _b.TgemmError(st, fn.__name__)


def kv_append(cache: PagedCache, K: torch.Tensor, V: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
              starts: torch.Tensor = None, weights: torch.Tensor = None, stream=None) -> None:
    """Write the newest tokens' keys and values, [tokens, heads, dim], into the
    cache.  Sequence b brings tokens starts[b] .. starts[b + 1] - 1 (starts:
    int32 [batch + 1]; None: one token each), which lengths[b] counts already:
    its last token goes to position lengths[b] - 1.  weights (float32 [batch,
    heads, positions]) are set to zero there."""
    index = cache._index
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    shape, sk, dtype = K.shape, K.stride(), K.dtype
    if len(shape) != 3 or V.shape != shape or shape[1] != cache.heads or shape[2] != cache.dim:
        raise ValueError("K and V must be [tokens, heads, dim] of the cache's heads and dim")
    if sk[2] != 1 or V.stride() != sk:
        raise ValueError("K and V must share strides, with unit stride of dim")
    if dtype not in cache._dtypes or V.dtype is not dtype:
        raise ValueError("K and V must be float16 or bfloat16, and the cache's dtype unless that is e4m3")
    if K.get_device() != index or V.get_device() != index:
        raise ValueError("K and V must be on the cache's device")
    if starts is not None:
        start = _vector("starts", starts, batch + 1, index)
    elif shape[0] == batch:
        start = 0
    else:
        raise ValueError("without starts every sequence brings one token")
    w = _NO_WEIGHTS if weights is None else _weights("weights", weights, batch, cache.heads, index)
    _launch(index, stream, _b.tgemm_kv_append,
            _append(cache._address, pages, length, width, stride, batch, *w, K.data_ptr(), V.data_ptr(), start,
                    shape[0], sk[0], sk[1], _DT[dtype]))


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
    index = cache._index
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    shape, sq, so, dtype = Q.shape, Q.stride(), O.stride(), Q.dtype
    if len(shape) != 3 or O.shape != shape or shape[0] != batch or shape[2] != cache.dim or shape[1] % cache.heads:
        raise ValueError("Q and O must be [batch, q_heads, dim], q_heads a multiple of the cache's heads")
    if sq[2] != 1 or so[2] != 1:
        raise ValueError("Q and O need unit stride of dim")
    if dtype not in cache._dtypes or O.dtype is not dtype:
        raise ValueError("Q and O must be float16 or bfloat16, and the cache's dtype unless that is e4m3")
    if Q.get_device() != index or O.get_device() != index:
        raise ValueError("Q and O must be on the cache's device")
    w = _NO_WEIGHTS if weights is None else _weights("weights", weights, batch, cache.heads, index)
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    if workspace is None:
        with torch.cuda.stream(stream):   # the zeros belong to the stream that uses them
            workspace = attention_decode_workspace(Q, cache, page_table, weights is not None)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the cache's device")
    _launch(index, stream, _b.tgemm_attention_decode,
            _decode(cache._address, pages, length, width, stride, batch, *w, Q.data_ptr(), O.data_ptr(), shape[1],
                    sq[0], sq[1], so[0], so[1], window, cache.dim ** -0.5 if scale is None else scale, cap,
                    workspace.data_ptr(), workspace.nbytes, _DT[dtype]))
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
    index, heads = cache._index, cache.heads
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    to_pages, to_width, to_stride, to_batch = _table(to_page_table, index)
    if to_batch != batch or to_cache._index != index or to_cache.dtype is not cache.dtype or to_cache.heads != heads or (
            to_cache.dim != cache.dim):
        raise ValueError("both caches must share dtype, heads, dim and device, both page tables the batch")
    shape = kept.shape
    if len(shape) != 3 or shape[0] != batch or shape[1] != heads or kept.dtype is not torch.int32 or (
            not kept.is_contiguous()) or kept.get_device() != index:
        raise ValueError("kept must be a contiguous int32 [batch, heads, keep] tensor on the cache's device")
    to_length = _vector("to_lengths", to_lengths, batch, index)
    w = _weights("weights", weights, batch, heads, index)
    to_w = _weights("to_weights", to_weights, batch, heads, index)
    if to_w[1] < shape[2]:
        raise ValueError("to_weights must hold at least keep positions")
    _launch(index, stream, _b.tgemm_kv_evict,
            _evict(cache._address, pages, length, width, stride, batch, *w, to_cache._address, to_pages, 0, to_width,
                   to_stride, batch, *to_w, kept.data_ptr(), to_length, shape[2], recent))
