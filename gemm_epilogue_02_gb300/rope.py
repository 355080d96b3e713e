"""Norms of queries and keys for each head with the position rotation in the same
pass, and its gradient.

The computation lives in the CUDA library (csrc/rope.cuh, C ABI in
include/tgemm.h); this module checks torch tensors and packs their addresses and
sizes into the calls' argument structures, as kv.py does.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _binding as _b
from .kv import _DT, _I32, _launch

_forward, _backward = _b.QK_NORM_ROPE_ARGS.pack, _b.QK_NORM_ROPE_BACKWARD_ARGS.pack
# 2^192 / (2 pi), rounded down
_PER_TURN = 2 ** 191 * 10 ** 75 // 3141592653589793238462643383279502884197169399375105820974944592307816406286
_NO_ROWS = (0, 0, 0)
_F32 = torch.float32


class Rotary:
    """A rotation of heads by position: pair i turns by `frequencies[i]` radians per
    position (any sequence of numbers) of axis axes[i] (None: one axis for all).
    The pairs are elements i and i + len(frequencies) of a head, or, interleaved,
    2 i and 2 i + 1; elements past them stay.  The object holds the frequencies as
    the library takes them, as fractions of a turn in 64 bits, in host memory: one
    serves any device."""

    def __init__(self, frequencies, axes=None, interleaved: bool = False):
        rates = [float(f) for f in frequencies]
        if axes is not None:
            axes = [int(a) for a in axes]
            if len(axes) != len(rates) or any(a < 0 or a > 31 for a in axes):
                raise ValueError("axes must name an axis, 0 to 31, for each frequency")
        if not interleaved and len(rates) % 4:
            raise ValueError("pairs that are not interleaved must be a multiple of 4")
        if not all(abs(f) < 2.0 ** 64 for f in rates):
            raise ValueError("frequencies must be finite and below 2^64")
        # f = m 2^e, m a whole number below 2^53: f / (2 pi) * 2^64, rounded down and without its whole turns
        turns = []
        for f in rates:
            m, e = math.frexp(f)
            turns.append((int(m * 2.0 ** 53) * _PER_TURN >> 181 - e) & 0xFFFFFFFFFFFFFFFF)
        self.pairs, self.interleaved, self.axes = len(rates), bool(interleaved), 1 if axes is None and rates else max(axes or (), default=-1) + 1
        self._turns = (ctypes.c_uint64 * max(1, len(rates)))(*turns)
        self._axes = None if axes is None else (ctypes.c_int32 * max(1, len(rates)))(*axes)
        c = _b.RotaryStruct()
        c.turns, c.axes = ctypes.addressof(self._turns), None if axes is None else ctypes.addressof(self._axes)
        c.pairs, c.interleaved = self.pairs, int(self.interleaved)
        self._struct = c
        self._address = ctypes.addressof(c)


_BAD_ROWS = "{} must be [tokens, heads, dim] of its input's shape and dtype with unit stride of dim"


def _refuse(Q, K, positions, rotary, eps, weights):
    """Says what is wrong with arguments that _common() does not take."""
    if Q.dim() != 3 or Q.dtype not in _DT or Q.stride(2) != 1:
        raise ValueError("Q must be float16 or bfloat16 [tokens, q_heads, dim] with unit stride of dim")
    if K is not None and (K.dim() != 3 or K.shape[0] != Q.shape[0] or K.shape[2] != Q.shape[2] or K.dtype is not Q.dtype
                          or K.stride(2) != 1):
        raise ValueError("K must be [tokens, k_heads, dim] of Q's tokens, dim and dtype with unit stride of dim")
    for w in weights:
        if w is not None and (w.shape != Q.shape[2:] or not w.is_contiguous() or w.dtype not in (Q.dtype, _F32)):
            raise ValueError("weights must be contiguous [dim] tensors, float32 or of Q's dtype")
    if eps is None and any(w is not None for w in weights):
        raise ValueError("weights go with the norm: eps must be a number")
    if rotary is None:
        raise ValueError("neither a norm nor a rotation")
    if 2 * rotary.pairs > Q.shape[2]:
        raise ValueError("the rotation has more pairs than a head")
    if positions is None:
        raise ValueError("a rotation needs positions")
    raise ValueError("q_weight and k_weight must share dtype, and positions be int32 [axes, tokens] (or [tokens]) with unit stride "
                     "of tokens")


def _common(Q, K, positions, rotary, q_weight, k_weight, eps, shift):
    """(Q's shape, dtype and row arguments, K's shape and row arguments, the arguments after the rows).  Written out, as a
    call's time is the host's where rows are few: every attribute of a tensor is read once, and it is left to the library
    to find tensors that are not on its device."""
    shape, dtype, stride = Q.shape, Q.dtype, Q.stride()
    code = _DT.get(dtype)
    if len(shape) != 3 or stride[2] != 1 or code is None:
        _refuse(Q, K, positions, rotary, eps, (q_weight, k_weight))
    tokens, q_heads, dim = shape
    q = (Q.data_ptr(), stride[0], stride[1])
    good = True
    if K is None:
        k, k_shape, k_heads = _NO_ROWS, None, 0
    else:
        k_shape, stride = K.shape, K.stride()
        if len(k_shape) != 3:
            _refuse(Q, K, positions, rotary, eps, (q_weight, k_weight))
        k_tokens, k_heads, k_dim = k_shape
        good = k_tokens == tokens and k_dim == dim and K.dtype is dtype and stride[2] == 1
        k = (K.data_ptr(), stride[0], stride[1])
    kind, qw, kw = None, 0, 0
    if q_weight is not None:
        kind = q_weight.dtype
        good = good and q_weight.dim() == 1 and q_weight.numel() == dim and q_weight.is_contiguous() and eps is not None
        qw = q_weight.data_ptr()
    if k_weight is not None:
        good = good and k_weight.dim() == 1 and k_weight.numel() == dim and k_weight.is_contiguous() and eps is not None and (
            kind is None or k_weight.dtype is kind)
        kind = k_weight.dtype
        kw = k_weight.data_ptr()
    if kind is not None and kind is not dtype and kind is not _F32:
        good = False
    if rotary is None:
        where = axis_stride = axes = plan = 0
        good = good and eps is not None
    elif positions is None:
        good = False
    else:
        plan, axes, stride, p = rotary._address, rotary.axes, positions.stride(), positions.shape
        if len(p) == 2:
            good = good and p[1] == tokens and p[0] >= axes and (stride[1] == 1 or tokens <= 1)
        else:
            good = good and len(p) == 1 and p[0] == tokens and axes <= 1 and (stride[0] == 1 or tokens <= 1)
        good = good and positions.dtype is _I32 and 2 * rotary.pairs <= dim
        where, axis_stride = positions.data_ptr(), stride[0]
    if not good:
        _refuse(Q, K, positions, rotary, eps, (q_weight, k_weight))
    return shape, dtype, q, k_shape, k, (qw, kw, where, axis_stride, axes, tokens, q_heads, k_heads, dim, shift, plan,
                                         kind is _F32, eps is not None, eps or 0.0, code)


def _rows(name, t, shape, dtype):
    """The row arguments of a tensor of that shape and dtype."""
    if t is None or t.dtype is not dtype or t.shape != shape:
        raise ValueError(_BAD_ROWS.format(name))
    stride = t.stride()
    if stride[2] != 1:
        raise ValueError(_BAD_ROWS.format(name))
    return t.data_ptr(), stride[0], stride[1]


def qk_norm_rope(Q: torch.Tensor, K: torch.Tensor, positions: torch.Tensor, rotary: Rotary, Q_out: torch.Tensor,
                 K_out: torch.Tensor, q_weight: torch.Tensor = None, k_weight: torch.Tensor = None, eps: float = 1e-6,
                 shift: int = 0, stream=None) -> None:
    """Q_out and K_out = the rows of Q [tokens, q_heads, dim] and K [tokens, k_heads,
    dim] (None: queries alone), each divided by the root of its mean square (plus
    eps; eps=None: no norm), times its weights ([dim], of Q's dtype or float32;
    None: ones), and turned by `rotary` (None: not turned) at the token's positions
    (int32 [axes, tokens] or [tokens], plus `shift`: with the lengths that kv_append()
    takes, shift=-1).  Q_out may be Q and K_out K."""
    shape, dtype, q, k_shape, k, rest = _common(Q, K, positions, rotary, q_weight, k_weight, eps, shift)
    if (K is None) != (K_out is None):
        raise ValueError("K and K_out go together")
    k_out = _NO_ROWS if K is None else _rows("K_out", K_out, k_shape, dtype)
    _launch(Q.get_device(), stream, _b.tgemm_qk_norm_rope, _forward(*q, *k, *_rows("Q_out", Q_out, shape, dtype), *k_out, *rest))


def qk_norm_rope_backward_workspace(Q: torch.Tensor, K: torch.Tensor = None) -> torch.Tensor:
    """A workspace for qk_norm_rope_backward() with weights' gradients: zeroed device
    memory, to be kept between calls, of any number of tokens and heads.  Calls that
    may overlap on the GPU need one each."""
    return torch.zeros(_b.tgemm_qk_norm_rope_backward_workspace(Q.shape[2]), dtype=torch.uint8, device=Q.device)


def qk_norm_rope_backward(Q_out_grad: torch.Tensor, K_out_grad: torch.Tensor, Q: torch.Tensor, K: torch.Tensor,
                          positions: torch.Tensor, rotary: Rotary, Q_grad: torch.Tensor, K_grad: torch.Tensor,
                          q_weight: torch.Tensor = None, k_weight: torch.Tensor = None, q_weight_grad: torch.Tensor = None,
                          k_weight_grad: torch.Tensor = None, eps: float = 1e-6, shift: int = 0,
                          workspace: torch.Tensor = None, stream=None) -> None:
    """The gradients of qk_norm_rope(): Q_grad and K_grad (which may be Q_out_grad
    and K_out_grad, or Q and K) from those of its outputs, and the weights'
    (float32 [dim], written; None: not wanted).  Sums are in a fixed order.  Without
    a workspace one is allocated and zeroed for the call if weights' gradients are
    wanted."""
    shape, dtype, q, k_shape, k, rest = _common(Q, K, positions, rotary, q_weight, k_weight, eps, shift)
    index = Q.get_device()
    if K is None:
        if K_out_grad is not None or K_grad is not None:
            raise ValueError("K, K_out_grad and K_grad go together")
        k_grad = k_out_grad = _NO_ROWS
    else:
        k_grad, k_out_grad = _rows("K_grad", K_grad, k_shape, dtype), _rows("K_out_grad", K_out_grad, k_shape, dtype)
    dw = [0, 0]
    for i, t in enumerate((q_weight_grad, k_weight_grad)):
        if t is not None:
            if eps is None or t.dtype is not _F32 or t.dim() != 1 or t.numel() != shape[2] or not t.is_contiguous():
                raise ValueError("weights' gradients go with the norm and must be contiguous float32 [dim] tensors")
            dw[i] = t.data_ptr()
    space = room = 0
    if q_weight_grad is not None or k_weight_grad is not None:
        if index < 0:
            raise ValueError("Q must be on a CUDA device")
        if workspace is None:
            with torch.cuda.stream(stream):   # the zeros belong to the stream that uses them
                workspace = qk_norm_rope_backward_workspace(Q)
        elif not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        space, room = workspace.data_ptr(), workspace.nbytes
    _launch(index, stream, _b.tgemm_qk_norm_rope_backward,
            _backward(*q, *k, *_rows("Q_grad", Q_grad, shape, dtype), *k_grad, *rest,
                      *_rows("Q_out_grad", Q_out_grad, shape, dtype), *k_out_grad, dw[0], dw[1], space, room))
