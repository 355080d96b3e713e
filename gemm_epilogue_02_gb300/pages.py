"""The paged cache's pages: bounds of the keys on them, the choice of pages by a
query, and growing, forking, freeing and compacting.

The computation lives in the CUDA library (csrc/page_bounds.cuh, csrc/page_pool.cuh,
C ABI in include/tgemm.h); this module checks torch tensors and packs their
addresses and sizes into the calls' argument structures, as kv.py does.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from .kv import _DT, PagedCache, _launch, _table, _vector

_bounds, _select, _grow = _b.KV_BOUNDS_ARGS.pack, _b.KV_SELECT_ARGS.pack, _b.KV_GROW_ARGS.pack
_fork, _free, _compact = _b.KV_FORK_ARGS.pack, _b.KV_FREE_ARGS.pack, _b.KV_COMPACT_ARGS.pack


class PageBounds:
    """Each page's bounds of its keys: bounds int8 [pages, heads, 2, dim] (least,
    largest) and scale float32 [pages, heads], both contiguous; a key k of channel
    d lies in scale * bounds[page, head, 0, d] .. scale * bounds[page, head, 1, d].
    The object keeps the tensors and their description; it owns nothing else."""

    def __init__(self, bounds: torch.Tensor, scale: torch.Tensor):
        if bounds.dim() != 4 or bounds.shape[2] != 2 or bounds.dtype is not torch.int8 or not bounds.is_contiguous():
            raise ValueError("bounds must be a contiguous int8 [pages, heads, 2, dim] tensor")
        if scale.dtype is not torch.float32 or scale.shape != bounds.shape[:2] or not scale.is_contiguous() or (
                scale.device != bounds.device):
            raise ValueError("scale must be a contiguous float32 [pages, heads] tensor on the bounds' device")
        self.bounds, self.scale = bounds, scale
        self._shape = (bounds.shape[0], bounds.shape[1], bounds.shape[3])
        self._index = bounds.get_device()
        c = _b.KvPageBounds()
        c.bounds, c.scale = bounds.data_ptr() or None, scale.data_ptr() or None
        self._struct = c
        self._address = ctypes.addressof(c)


def _check_bounds(bounds, cache):
    if bounds._shape != (cache.pages, cache.heads, cache.dim) or bounds._index != cache._index:
        raise ValueError("the bounds must be of the cache's pages, heads and dim and on its device")
    return bounds._address


def _uses(name, t, cache):
    return _vector(name, t, cache.pages, cache._index)


def kv_bounds(cache: PagedCache, bounds: PageBounds, page_table: torch.Tensor, lengths: torch.Tensor,
              starts: torch.Tensor = None, stream=None) -> None:
    """Write the bounds of the pages that the newest tokens complete: sequence b
    has brought starts[b + 1] - starts[b] of them (starts: int32 [batch + 1]; None:
    one token each), which lengths[b] counts already, as after kv_append()."""
    index = cache._index
    address = _check_bounds(bounds, cache)
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    start = 0 if starts is None else _vector("starts", starts, batch + 1, index)
    _launch(index, stream, _b.tgemm_kv_bounds,
            _bounds(cache._address, address, pages, length, width, stride, batch, start, _DT.get(cache.dtype, 0)))


def kv_select(Q: torch.Tensor, cache: PagedCache, bounds: PageBounds, page_table: torch.Tensor, lengths: torch.Tensor,
              to_page_table: torch.Tensor, to_lengths: torch.Tensor, first: int = 0, recent: int = 1, stream=None) -> None:
    """Choose the pages that matter to each key head's queries: of a sequence's
    pages at most keep = to_page_table.shape[2] stay, the first `first`, the last
    `recent` and those between them whose bounds allow the largest product with
    one of the head's queries, as rounded to 8 bits of its largest element.  Q is [batch, q_heads, dim].  Written are
    to_page_table (int32 [batch, heads, keep], in order of position, -1 past them)
    and to_lengths (int32 [batch], the positions on them), for attention_decode()."""
    index = cache._index
    address = _check_bounds(bounds, cache)
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    shape, sq, dtype = Q.shape, Q.stride(), Q.dtype
    if len(shape) != 3 or shape[0] != batch or shape[2] != cache.dim or shape[1] % cache.heads or sq[2] != 1:
        raise ValueError("Q must be [batch, q_heads, dim] with unit stride of dim, q_heads a multiple of the cache's heads")
    if dtype not in cache._dtypes:
        raise ValueError("Q must be float16 or bfloat16, and the cache's dtype unless that is e4m3")
    to, st = to_page_table.shape, to_page_table.stride()
    if len(to) != 3 or to[0] != batch or to[1] != cache.heads or to_page_table.dtype is not torch.int32 or (st[2] != 1 and to[2] > 1):
        raise ValueError("to_page_table must be int32 [batch, heads, keep] with unit stride of keep")
    if Q.get_device() != index or to_page_table.get_device() != index:
        raise ValueError("Q and to_page_table must be on the cache's device")
    to_length = _vector("to_lengths", to_lengths, batch, index)
    _launch(index, stream, _b.tgemm_kv_select,
            _select(cache._address, address, pages, length, width, stride, batch, Q.data_ptr(), shape[1], sq[0], sq[1],
                    to_page_table.data_ptr(), to_length, st[0], st[1], to[2], first, recent, _DT[dtype]))


def kv_grow(cache: PagedCache, uses: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
            tokens: torch.Tensor = None, stream=None) -> None:
    """Make room for new tokens: lengths[b] grows by tokens[b] (int32 [batch]; None:
    one each) and the page table by the pages that this takes, the lowest free ones
    in the order of the sequences.  uses (int32 [pages]) counts the sequences that
    hold each page."""
    index = cache._index
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    fresh = 0 if tokens is None else _vector("tokens", tokens, batch, index)
    _launch(index, stream, _b.tgemm_kv_grow,
            _grow(cache._address, _uses("uses", uses, cache), pages, length, width, stride, batch, fresh))


def kv_fork(cache: PagedCache, uses: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor, parents: torch.Tensor,
            to_page_table: torch.Tensor, to_lengths: torch.Tensor, stream=None) -> None:
    """Child c takes over the positions of sequence parents[c] (int32 [children];
    -1: none): full pages are shared, the rows of a last, partly filled page are
    copied to a free page.  to_page_table and to_lengths may be other rows of
    page_table and lengths, as long as no child is a parent; what the children held
    before is to be freed first (kv_free)."""
    index = cache._index
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    to_pages, to_width, to_stride, children = _table(to_page_table, index)
    to_length = _vector("to_lengths", to_lengths, children, index)
    _launch(index, stream, _b.tgemm_kv_fork,
            _fork(cache._address, _uses("uses", uses, cache), pages, length, width, stride, batch,
                  _vector("parents", parents, children, index), to_pages, to_length, to_width, to_stride, children))


def kv_free(cache: PagedCache, uses: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor, stream=None) -> None:
    """The sequences give their pages back: uses goes down by one on each, lengths
    become 0 (a length that its list cannot hold stays, as does what it counts)."""
    index = cache._index
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    _launch(index, stream, _b.tgemm_kv_free,
            _free(cache._address, _uses("uses", uses, cache), pages, length, width, stride, batch))


def kv_compact_workspace(cache: PagedCache) -> torch.Tensor:
    """A workspace for kv_compact(), with any contents.  Calls that may overlap on the GPU need one each."""
    return torch.empty(_b.tgemm_kv_compact_workspace(cache.pages), dtype=torch.uint8, device=cache.device)


def kv_compact(cache: PagedCache, uses: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
               to_page_table: torch.Tensor, to_uses: torch.Tensor, in_use: torch.Tensor, bounds: PageBounds = None,
               workspace: torch.Tensor = None, stream=None) -> None:
    """Move the pages in use below their number n, so that the pool is free from
    page n on: those above go, in order, to the free ones below, with scales and
    bounds.  page_table has all sequences that hold pages.  Written are
    to_page_table (the new numbers), to_uses (int32 [pages]) and in_use (int32 [1],
    n); to_page_table may be page_table and to_uses uses.  Without a workspace one
    is allocated for the call."""
    index = cache._index
    pages, width, stride, batch = _table(page_table, index)
    length = _vector("lengths", lengths, batch, index)
    to_pages, to_width, to_stride, to_batch = _table(to_page_table, index)
    if to_batch != batch or to_width < width:
        raise ValueError("to_page_table must have the sequences of page_table, and room for their lists")
    address = 0 if bounds is None else _check_bounds(bounds, cache)
    count, to_count, total = _uses("uses", uses, cache), _uses("to_uses", to_uses, cache), _vector("in_use", in_use, 1, index)
    if index < 0:
        raise ValueError("the cache must be on a CUDA device")
    if workspace is None:
        with torch.cuda.stream(stream):   # the memory belongs to the stream that uses it
            workspace = kv_compact_workspace(cache)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the cache's device")
    _launch(index, stream, _b.tgemm_kv_compact,
            _compact(cache._address, address, count, pages, length, width, stride, batch, to_pages, to_width, to_stride,
                     to_count, total, workspace.data_ptr(), workspace.nbytes))
