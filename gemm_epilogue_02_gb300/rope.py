"""Norms of queries and keys for each head with the position rotation in the same
pass, and its gradient.

The computation lives in the CUDA library (csrc/rope.cuh, C ABI in
include/tgemm.h); this module checks torch tensors and packs their addresses and
sizes into the calls' argument structures, as kv.py does.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from .kv import _DT, _launch

_forward, _backward = _b.QK_NORM_ROPE_ARGS.pack, _b.QK_NORM_ROPE_BACKWARD_ARGS.pack
# pi * 2^188 (3.14159265358979323846264338327950288419716939937510582097494), rounded.
_PI_188 = 314159265358979323846264338327950288419716939937510582097494 * 2 ** 188 // 10 ** 59
_NO_ROWS = (0, 0, 0)


class Rotary:
    """A rotation of heads by position: pair i turns by `frequencies[i]` radians per
    position (any sequence of numbers) of axis axes[i] (None: one axis for all).
    The pairs are elements i and i + len(frequencies) of a head, or, interleaved,
    2 i and 2 i + 1; elements past them stay.  The object holds the frequencies as
    the library takes them, as fractions of a turn in 64 bits, in host memory: one
    serves any device."""

    def __init__(self, frequencies, axes=None, interleaved: bool = False):
        rates = [float(f) for f in frequencies]
        axes = [0] * len(rates) if axes is None else [int(a) for a in axes]
        if len(axes) != len(rates) or any(a < 0 or a > 31 for a in axes):
            raise ValueError("axes must name an axis, 0 to 31, for each frequency")
        if not interleaved and len(rates) % 4:
            raise ValueError("pairs that are not interleaved must be a multiple of 4")
        try:
            ratios = [f.as_integer_ratio() for f in rates]
        except (OverflowError, ValueError):
            raise ValueError("frequencies must be finite") from None
        # f / (2 pi) * 2^64, towards minus infinity
        turns = [(n << 251) // (d * _PI_188) & 0xFFFFFFFFFFFFFFFF for n, d in ratios]
        self.pairs, self.interleaved, self.axes = len(rates), bool(interleaved), max(axes, default=-1) + 1
        self._turns = (ctypes.c_uint64 * max(1, len(rates)))(*turns)
        self._axes = (ctypes.c_int32 * max(1, len(rates)))(*axes)
        c = _b.RotaryStruct()
        c.turns, c.axes = ctypes.addressof(self._turns), ctypes.addressof(self._axes)
        c.pairs, c.interleaved = self.pairs, int(self.interleaved)
        self._struct = c
        self._address = ctypes.addressof(c)


def _rows(name, t, like, index):
    """(address, token stride, head stride) of rows of heads with the shape and dtype of `like`."""
    stride = t.stride()
    if t.shape != like.shape or t.dtype is not like.dtype or stride[2] != 1 or t.get_device() != index:
        raise ValueError(f"{name} must be [tokens, heads, dim] of its input's shape, dtype and device with unit stride of dim")
    return t.data_ptr(), stride[0], stride[1]


def _common(Q, K, positions, rotary, q_weight, k_weight, eps, shift):
    """(device index, heads of K, the arguments after the rows)."""
    index, shape, dtype = Q.get_device(), Q.shape, Q.dtype
    if len(shape) != 3 or dtype not in _DT or Q.stride(2) != 1:
        raise ValueError("Q must be float16 or bfloat16 [tokens, q_heads, dim] with unit stride of dim")
    k_heads = 0
    if K is not None:
        if K.dim() != 3 or K.shape[0] != shape[0] or K.shape[2] != shape[2] or K.dtype is not dtype or K.stride(2) != 1 or (
                K.get_device() != index):
            raise ValueError("K must be [tokens, k_heads, dim] of Q's tokens, dim, dtype and device with unit stride of dim")
        k_heads = K.shape[1]
    wide = None
    weights = []
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            weights.append(0)
            continue
        if w.dtype is not dtype and w.dtype is not torch.float32:
            raise ValueError(f"{name} must be float32 or of Q's dtype")
        if w.dim() != 1 or w.numel() != shape[2] or not w.is_contiguous() or w.get_device() != index:
            raise ValueError(f"{name} must be a contiguous [dim] tensor on Q's device")
        if wide is not None and wide != (w.dtype is torch.float32):
            raise ValueError("q_weight and k_weight must share dtype")
        wide = w.dtype is torch.float32
        weights.append(w.data_ptr())
    if eps is None and (q_weight is not None or k_weight is not None):
        raise ValueError("weights go with the norm: eps must be a number")
    where, axis_stride, axes, plan = 0, 0, 0, 0
    if rotary is not None:
        plan, axes = rotary._address, rotary.axes
        if 2 * rotary.pairs > shape[2]:
            raise ValueError("the rotation has more pairs than a head")
        if positions is None:
            raise ValueError("a rotation needs positions")
        p = positions.unsqueeze(0) if positions.dim() == 1 else positions
        if p.dtype is not torch.int32 or p.dim() != 2 or p.shape[1] != shape[0] or p.shape[0] < axes or (
                p.stride(1) != 1 and shape[0] > 1) or p.get_device() != index:
            raise ValueError("positions must be int32 [axes, tokens] (or [tokens]) on Q's device with unit stride of tokens")
        where, axis_stride = p.data_ptr(), p.stride(0)
    elif eps is None:
        raise ValueError("neither a norm nor a rotation")
    return index, k_heads, (weights[0], weights[1], where, axis_stride, axes, shape[0], shape[1], k_heads, shape[2], shift, plan,
                            int(bool(wide)), int(eps is not None), 0.0 if eps is None else eps, _DT[dtype])


def qk_norm_rope(Q: torch.Tensor, K: torch.Tensor, positions: torch.Tensor, rotary: Rotary, Q_out: torch.Tensor,
                 K_out: torch.Tensor, q_weight: torch.Tensor = None, k_weight: torch.Tensor = None, eps: float = 1e-6,
                 shift: int = 0, stream=None) -> None:
    """Q_out and K_out = the rows of Q [tokens, q_heads, dim] and K [tokens, k_heads,
    dim] (None: queries alone), each divided by the root of its mean square (plus
    eps; eps=None: no norm), times its weights ([dim], of Q's dtype or float32;
    None: ones), and turned by `rotary` (None: not turned) at the token's positions
    (int32 [axes, tokens] or [tokens], plus `shift`: with the lengths that kv_append()
    takes, shift=-1).  Q_out may be Q and K_out K."""
    index, k_heads, rest = _common(Q, K, positions, rotary, q_weight, k_weight, eps, shift)
    if (K is None) != (K_out is None):
        raise ValueError("K and K_out go together")
    q, q_out = _rows("Q", Q, Q, index), _rows("Q_out", Q_out, Q, index)
    k, k_out = (_NO_ROWS, _NO_ROWS) if K is None else (_rows("K", K, K, index), _rows("K_out", K_out, K, index))
    _launch(index, stream, _b.tgemm_qk_norm_rope, _forward(*q, *k, *q_out, *k_out, *rest))


def qk_norm_rope_backward_workspace(Q: torch.Tensor, K: torch.Tensor = None) -> torch.Tensor:
    """A workspace for qk_norm_rope_backward() with weights' gradients, with any
    contents.  Calls that may overlap on the GPU need one each."""
    return torch.empty(_b.tgemm_qk_norm_rope_backward_workspace(Q.shape[2]), dtype=torch.uint8, device=Q.device)


def qk_norm_rope_backward(Q_out_grad: torch.Tensor, K_out_grad: torch.Tensor, Q: torch.Tensor, K: torch.Tensor,
                          positions: torch.Tensor, rotary: Rotary, Q_grad: torch.Tensor, K_grad: torch.Tensor,
                          q_weight: torch.Tensor = None, k_weight: torch.Tensor = None, q_weight_grad: torch.Tensor = None,
                          k_weight_grad: torch.Tensor = None, eps: float = 1e-6, shift: int = 0,
                          workspace: torch.Tensor = None, stream=None) -> None:
    """The gradients of qk_norm_rope(): Q_grad and K_grad (which may be Q_out_grad
    and K_out_grad, or Q and K) from those of its outputs, and the weights'
    (float32 [dim], written; None: not wanted).  Sums are in a fixed order.  Without
    a workspace one is allocated for the call if weights' gradients are wanted."""
    index, k_heads, rest = _common(Q, K, positions, rotary, q_weight, k_weight, eps, shift)
    if any((t is None) != (K is None) for t in (K_out_grad, K_grad)):
        raise ValueError("K, K_out_grad and K_grad go together")
    grads = []
    for name, t in (("q_weight_grad", q_weight_grad), ("k_weight_grad", k_weight_grad)):
        if t is not None and (t.dtype is not torch.float32 or t.dim() != 1 or t.numel() != Q.shape[2] or not t.is_contiguous()
                              or t.get_device() != index):
            raise ValueError(f"{name} must be a contiguous float32 [dim] tensor on Q's device")
        grads.append(0 if t is None else t.data_ptr())
    if eps is None and any(grads):
        raise ValueError("weights go with the norm: eps must be a number")
    rows = [_rows(n, t, Q, index) for n, t in (("Q", Q), ("Q_grad", Q_grad), ("Q_out_grad", Q_out_grad))]
    rows += [_NO_ROWS] * 3 if K is None else [_rows(n, t, K, index)
                                              for n, t in (("K", K), ("K_grad", K_grad), ("K_out_grad", K_out_grad))]
    if index < 0:
        raise ValueError("Q must be on a CUDA device")
    if not any(grads):
        workspace = None
    elif workspace is None:
        with torch.cuda.stream(stream):   # the memory belongs to the stream that uses it
            workspace = qk_norm_rope_backward_workspace(Q)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on Q's device")
    _launch(index, stream, _b.tgemm_qk_norm_rope_backward,
            _backward(*rows[0], *rows[3], *rows[1], *rows[4], *rest, *rows[2], *rows[5], *grads,
                      0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes))
