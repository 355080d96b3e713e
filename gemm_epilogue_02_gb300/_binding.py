"""Thin ctypes binding of the C ABI in include/tgemm.h.

Argument marshalling only: every step of the computation runs in the CUDA
library.  There is no CPU fallback; if the library cannot be loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

TGEMM_F16, TGEMM_BF16 = 0, 1
TGEMM_EPI_NONE, TGEMM_EPI_RELU, TGEMM_EPI_BIAS, TGEMM_EPI_BIAS_RELU = 0, 1, 2, 3
TGEMM_EPI_GELU, TGEMM_EPI_BIAS_GELU = 4, 5
STATUS = {0: "TGEMM_OK", 1: "TGEMM_ERR_INVALID_ARG", 2: "TGEMM_ERR_ALIGNMENT",
          3: "TGEMM_ERR_UNSUPPORTED_DEVICE", 4: "TGEMM_ERR_ALIAS", 5: "TGEMM_ERR_CUDA",
          6: "TGEMM_ERR_TIMEOUT", 7: "TGEMM_ERR_SCRATCH_LIMIT", 8: "TGEMM_ERR_DEBUG_CHECK",
          9: "TGEMM_ERR_CACHE"}
EXPORTED = ("tgemm_run", "tgemm_run_ex", "tgemm_run_host", "tgemm_status_string",
            "tgemm_last_device_status", "tgemm_version", "tgemm_run_noalloc", "tgemm_plan",
            "tgemm_attention_fwd", "tgemm_debug_last_check", "tgemm_kv_append", "tgemm_attention_decode",
            "tgemm_attention_decode_workspace", "tgemm_kv_evict", "tgemm_attention_decode_lists", "tgemm_kv_bounds",
            "tgemm_kv_select", "tgemm_kv_grow", "tgemm_kv_fork", "tgemm_kv_free", "tgemm_kv_compact",
            "tgemm_kv_compact_workspace", "tgemm_qk_norm_rope", "tgemm_qk_norm_rope_backward",
            "tgemm_qk_norm_rope_backward_workspace")
PLAN_FIELDS = ("bn", "cg", "stages", "tiles", "groups", "split_k", "split_first", "narrow_first",
               "narrow_parts", "units")
NOALLOC_SCRATCH_BYTES = 64 << 20

_lock = threading.Lock()
_lib = None
_debug_lib = None


class KvCache(ctypes.Structure):
    """tgemm_kv_cache."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
                + [(n, ctypes.c_int64) for n in ("pages", "page_stride", "slot_stride", "head_stride",
                                                 "scale_page_stride", "scale_slot_stride", "scale_head_stride")]
                + [(n, ctypes.c_int32) for n in ("page_size", "heads", "dim", "e4m3")])


class KvPageBounds(ctypes.Structure):
    """tgemm_kv_page_bounds."""
    _fields_ = [("bounds", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class RotaryStruct(ctypes.Structure):
    """tgemm_rotary."""
    _fields_ = [("turns", ctypes.c_void_p), ("axes", ctypes.c_void_p), ("pairs", ctypes.c_int64), ("interleaved", ctypes.c_int64)]


# The argument structures of the calls below, as struct.pack formats (every
# field takes 8 bytes): pointers and sizes Q / q, real numbers d.
_SEQUENCES = "QQqqq"          # pages, lengths, pages_width, pages_stride, batch
_WEIGHTS = "Qqqq"             # data, width, batch_stride, head_stride
KV_APPEND_ARGS = struct.Struct("=Q" + _SEQUENCES + _WEIGHTS + "QQQqqqq")
ATTENTION_DECODE_ARGS = struct.Struct("=Q" + _SEQUENCES + _WEIGHTS + "QQqqqqqqddQqq")
KV_EVICT_ARGS = struct.Struct("=Q" + _SEQUENCES + _WEIGHTS + "Q" + _SEQUENCES + _WEIGHTS + "QQqq")
_LISTS = "QQqqq"              # pages, lengths, width, stride, batch
KV_BOUNDS_ARGS = struct.Struct("=QQ" + _SEQUENCES + "Qq")
KV_SELECT_ARGS = struct.Struct("=QQ" + _SEQUENCES + "QqqqQQqqqqqq")
KV_GROW_ARGS = struct.Struct("=QQ" + _LISTS + "Q")
KV_FORK_ARGS = struct.Struct("=QQ" + _SEQUENCES + "Q" + _LISTS)
KV_FREE_ARGS = struct.Struct("=QQ" + _LISTS)
KV_COMPACT_ARGS = struct.Struct("=QQQ" + _SEQUENCES + "QqqQQQq")
_ROWS = "Qqq"                 # data, token_stride, head_stride
_NORM_ROPE = 4 * _ROWS + "QQQqqqqqqqQqqdq"
QK_NORM_ROPE_ARGS = struct.Struct("=" + _NORM_ROPE)
QK_NORM_ROPE_BACKWARD_ARGS = struct.Struct("=" + _NORM_ROPE + 2 * _ROWS + "QQQq")


class TgemmError(RuntimeError):
    def __init__(self, status: int, where: str = "tgemm_run"):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(self.status, self.status)}")


def library_path() -> str:
    """The library load() uses: the debug build when TGEMM_DEBUG=1 is set."""
    return _build.DEBUG_LIB if os.environ.get("TGEMM_DEBUG") == "1" else _build.LIB


def _configure(lib: ctypes.CDLL) -> ctypes.CDLL:
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    for name in ("tgemm_run", "tgemm_run_host", "tgemm_run_noalloc"):
        f = getattr(lib, name)
        f.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, i64, i32, i32, p]
        f.restype = i32
    lib.tgemm_run_ex.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, i64, i32, i32, i32, i32, p]
    lib.tgemm_run_ex.restype = i32
    lib.tgemm_status_string.argtypes = [i32]
    lib.tgemm_status_string.restype = ctypes.c_char_p
    lib.tgemm_last_device_status.argtypes = []
    lib.tgemm_last_device_status.restype = i32
    lib.tgemm_debug_last_check.argtypes = []
    lib.tgemm_debug_last_check.restype = i32
    lib.tgemm_version.argtypes = []
    lib.tgemm_version.restype = i32
    lib.tgemm_plan.argtypes = [i64, i64, i64, i32, p]
    lib.tgemm_plan.restype = i32
    lib.tgemm_attention_fwd.argtypes = [p, p, p, p, i64, i64, i64, i64, i32, i32, p]
    lib.tgemm_attention_fwd.restype = i32
    for name in ("tgemm_kv_append", "tgemm_attention_decode", "tgemm_kv_evict", "tgemm_kv_bounds", "tgemm_kv_select",
                 "tgemm_kv_grow", "tgemm_kv_fork", "tgemm_kv_free", "tgemm_kv_compact", "tgemm_qk_norm_rope",
                 "tgemm_qk_norm_rope_backward"):
        f = getattr(lib, name)
        f.argtypes = [p, p]
        f.restype = i32
    lib.tgemm_attention_decode_workspace.argtypes = [i64, i64, i64, i64, i64, i32, p]
    lib.tgemm_attention_decode_workspace.restype = i32
    lib.tgemm_attention_decode_lists.argtypes = [p, i64, p]
    lib.tgemm_attention_decode_lists.restype = i32
    for name in ("tgemm_kv_compact_workspace", "tgemm_qk_norm_rope_backward_workspace"):
        f = getattr(lib, name)
        f.argtypes = [i64, p]
        f.restype = i32
    return lib


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libtgemm.so, or libtgemm_debug.so when TGEMM_DEBUG=1 is set at the
    first call (building them with nvcc if missing or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if build_if_missing:
            _build.build()
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing; run build() first")
        _lib = _configure(ctypes.CDLL(path))
        return _lib


def load_debug(build_if_missing: bool = True) -> ctypes.CDLL:
    """The debug build, loaded beside the library load() returns (its own
    device state); for tests that run both on the same inputs."""
    global _debug_lib
    with _lock:
        if _debug_lib is None:
            if build_if_missing:
                _build.build()
            if not os.path.exists(_build.DEBUG_LIB):
                raise RuntimeError(f"CUDA library {_build.DEBUG_LIB} is missing; run build() first")
            _debug_lib = _configure(ctypes.CDLL(_build.DEBUG_LIB))
        return _debug_lib


def tgemm_run(A: int, B: int, bias: int, C: int, M: int, N: int, K: int, lda: int, ldb: int,
              ldc: int, dtype: int, epilogue: int, stream: int = 0) -> int:
    """Raw C-ABI call with device pointers (ints); returns the status code."""
    lib = _lib if _lib is not None else load()
    return lib.tgemm_run(A or None, B or None, bias or None, C or None, M, N, K, lda, ldb, ldc,
                         dtype, epilogue, stream or None)


def tgemm_run_ex(A: int, B: int, bias: int, C: int, M: int, N: int, K: int, lda: int, ldb: int,
                 ldc: int, dtype: int, epilogue: int, transpose_a: int, transpose_b: int,
                 stream: int = 0) -> int:
    """Raw C-ABI call with either operand stored transposed; returns the status code."""
    return load().tgemm_run_ex(A or None, B or None, bias or None, C or None, M, N, K, lda, ldb, ldc,
                               dtype, epilogue, int(transpose_a), int(transpose_b), stream or None)


def tgemm_run_host(A: int, B: int, bias: int, C: int, M: int, N: int, K: int, lda: int, ldb: int,
                   ldc: int, dtype: int, epilogue: int, stream: int = 0) -> int:
    """Raw C-ABI call with host pointers (ints); returns the status code."""
    return load().tgemm_run_host(A or None, B or None, bias or None, C or None, M, N, K, lda, ldb,
                                 ldc, dtype, epilogue, stream or None)


def tgemm_run_noalloc(A: int, B: int, bias: int, C: int, M: int, N: int, K: int, lda: int,
                      ldb: int, ldc: int, dtype: int, epilogue: int, stream: int = 0) -> int:
    """Raw C-ABI call of the allocation-free variant (device pointers as ints).

    For callers that must not allocate GPU memory (memory reserved up front by
    another allocator, allocation-free latency loops): any operand repack uses
    the library's fixed 64 MiB device array instead of allocating; calls that
    may overlap on the GPU race on that array.  Returns the status code."""
    return load().tgemm_run_noalloc(A or None, B or None, bias or None, C or None, M, N, K, lda,
                                    ldb, ldc, dtype, epilogue, stream or None)


def tgemm_status_string(status: int) -> str:
    return load().tgemm_status_string(int(status)).decode()


def tgemm_last_device_status() -> int:
    return int(load().tgemm_last_device_status())


def tgemm_debug_last_check() -> int:
    """Id of the first failed device-side check of the debug build since the
    last call (0: none; -1: the loaded library is the release build)."""
    return int(load().tgemm_debug_last_check())


def tgemm_version() -> int:
    return int(load().tgemm_version())


def tgemm_plan(M: int, N: int, K: int, num_sms: int) -> dict:
    """The work plan of an M x N x K problem on `num_sms` SMs (host logic, no GPU)."""
    out = (ctypes.c_int32 * len(PLAN_FIELDS))()
    st = load().tgemm_plan(M, N, K, num_sms, ctypes.cast(out, ctypes.c_void_p))
    if st != 0:
        raise TgemmError(st, "tgemm_plan")
    return dict(zip(PLAN_FIELDS, (int(v) for v in out)))


def tgemm_attention_fwd(Q: int, K: int, V: int, O: int, batch: int, seq: int, heads: int, dim: int,
                        causal: int, dtype: int, stream: int = 0) -> int:
    return int(load().tgemm_attention_fwd(Q, K, V, O, batch, seq, heads, dim, int(causal), dtype, stream))


# The paged key-value cache: `args` are the bytes of the call's argument
# structure (KV_APPEND_ARGS.pack(...) and so on: the fields of include/tgemm.h
# in order, pointers as ints).
def tgemm_kv_append(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_kv_append(args, stream)


def tgemm_attention_decode(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_attention_decode(args, stream)


def tgemm_kv_evict(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_kv_evict(args, stream)


def tgemm_attention_decode_workspace(batch: int, q_heads: int, kv_heads: int, dim: int, positions: int,
                                     with_weights: bool) -> int:
    """Bytes of workspace of tgemm_attention_decode (host logic, no GPU)."""
    out = ctypes.c_int64()
    st = load().tgemm_attention_decode_workspace(batch, q_heads, kv_heads, dim, positions, int(with_weights),
                                                 ctypes.byref(out))
    if st != 0:
        raise TgemmError(st, "tgemm_attention_decode_workspace")
    return int(out.value)


def tgemm_attention_decode_lists(args: bytes, pages_head_stride: int, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_attention_decode_lists(args, pages_head_stride, stream)


def tgemm_kv_bounds(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_kv_bounds(args, stream)


def tgemm_kv_select(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_kv_select(args, stream)


def tgemm_kv_grow(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_kv_grow(args, stream)


def tgemm_kv_fork(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_kv_fork(args, stream)


def tgemm_kv_free(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_kv_free(args, stream)


def tgemm_kv_compact(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_kv_compact(args, stream)


def _workspace_bytes(name: str, n: int) -> int:
    out = ctypes.c_int64()
    st = getattr(load(), name)(n, ctypes.byref(out))
    if st != 0:
        raise TgemmError(st, name)
    return int(out.value)


def tgemm_kv_compact_workspace(pages: int) -> int:
    """Bytes of workspace of tgemm_kv_compact (host logic, no GPU)."""
    return _workspace_bytes("tgemm_kv_compact_workspace", pages)


# Head norms with the position rotation: `args` as above.
def tgemm_qk_norm_rope(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_qk_norm_rope(args, stream)


def tgemm_qk_norm_rope_backward(args: bytes, stream: int = 0) -> int:
    return (_lib if _lib is not None else load()).tgemm_qk_norm_rope_backward(args, stream)


def tgemm_qk_norm_rope_backward_workspace(dim: int) -> int:
    """Bytes of workspace of tgemm_qk_norm_rope_backward (host logic, no GPU)."""
    return _workspace_bytes("tgemm_qk_norm_rope_backward_workspace", dim)
