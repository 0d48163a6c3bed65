"""Python binding of libdetfold_attn, the decode step's attention over a paged
key-value cache (``include/detfold_attn.h``).

Argument marshalling only, as in the package itself: the functions keep the C
names; the compiled marshalling module checks the tensors that it is given
(device, type, shape, strides) and passes addresses on, the library checks the
rest. ``stream`` may be None (torch's current stream), a ``torch.cuda.Stream`` or a
raw handle. A negative status raises ``DetfoldError``; the ``status_*`` variants
return it instead. ``lib`` is the C ABI itself, through ctypes.

``PagedCache`` and ``Rope`` hold what a program keeps between calls: the cache
and the table of rotations, described once. They keep their tensors alive.
"""
from __future__ import annotations

import ctypes
import os

import torch  # noqa: F401  (the marshalling module uses its libraries)

from . import DetfoldError, STATUS, _build, _stream, detfold_status_string

__all__ = [
    "PagedCache", "Rope", "detfold_kv_append", "detfold_attn_decode", "detfold_attn_join",
    "detfold_attn_decode_workspace_bytes", "detfold_attn_last_cuda_error",
    "DETFOLD_F32", "DETFOLD_BF16", "DETFOLD_F16", "DETFOLD_ATTN_MAX_HEAD_DIM", "DETFOLD_ATTN_MAX_LEN",
    "DETFOLD_ATTN_MAX_COUNT",
]

DETFOLD_F32 = 0
DETFOLD_BF16 = 1
DETFOLD_F16 = 2
DETFOLD_ATTN_MAX_HEAD_DIM = 256
DETFOLD_ATTN_MAX_LEN = 1 << 30
DETFOLD_ATTN_MAX_COUNT = 1 << 20

ATTN_LIB_PATH = _build.ATTN_LIB
if not os.path.exists(ATTN_LIB_PATH):
    raise ImportError(
        f"libdetfold_attn.so is not built ({ATTN_LIB_PATH}); run "
        "`python -c 'import __graft_entry__ as g; g.build()'` first")

lib = ctypes.CDLL(ATTN_LIB_PATH)

try:
    from . import _attn_binding as _binding  # noqa: E402  (built and linked beside the library)
except ImportError as e:
    raise ImportError(f"the attention operators' binding does not load ({e}); "
                      "`python -c 'import __graft_entry__ as g; g.build()'` builds it and says what it lacks") from e

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int


class _Cache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("num_pages", _I64), ("page_stride", _I64), ("token_stride", _I64),
                ("head_stride", _I64), ("dtype", _INT), ("page_size", _INT), ("kv_heads", _INT),
                ("head_dim", _INT)]


class _Rope(ctypes.Structure):
    _fields_ = [("cos_sin", _P), ("positions", _I64), ("rot_dim", _INT), ("interleaved", _INT)]


lib.detfold_kv_append.argtypes = [_P, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _P,
                                  _I64, _I64, _INT, _P, _P]
lib.detfold_kv_append.restype = _INT
lib.detfold_attn_decode_workspace_bytes.argtypes = [_P, _INT, _INT, _I64]
lib.detfold_attn_decode_workspace_bytes.restype = _I64
lib.detfold_attn_decode.argtypes = [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _I64, _P, _INT, _INT,
                                    _I64, ctypes.c_float, _I64, _P, _I64, _P, _P]
lib.detfold_attn_decode.restype = _INT
lib.detfold_attn_join.argtypes = [_P, _P, _P, _P, _INT, _I64, _INT, _INT, _P]
lib.detfold_attn_join.restype = _INT
lib.detfold_attn_last_cuda_error.argtypes = []
lib.detfold_attn_last_cuda_error.restype = _INT

def _check(status: int, where: str) -> None:
    if status != 0:
        if status == STATUS["DETFOLD_ERR_CUDA"]:
            raise AttnError(status, where)
        raise DetfoldError(status, where)


class AttnError(DetfoldError):
    """A failed CUDA call of this library (its error value is kept apart from the fold library's)."""

    def __init__(self, status: int, where: str):
        RuntimeError.__init__(self, f"{where}: status {status}: {detfold_status_string(status)} "
                                    f"(cudaError {lib.detfold_attn_last_cuda_error()})")
        self.status = status


class PagedCache:
    """A paged cache: k and v of shape [pages, page_size, kv_heads, head_dim] with
    the same strides, any order of the first three dimensions (a view of a
    cache that is stored head by head, or of one buffer that holds both)."""

    def __init__(self, k, v):
        self._handle = _binding.cache(k, v)
        self.k, self.v = k, v


class Rope:
    """A table of rotations: cos_sin [positions, rot_dim] float32, cosines then
    sines. Pairs are elements (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved."""

    def __init__(self, cos_sin, interleaved: bool = False):
        self._handle = _binding.rope(cos_sin, interleaved)
        self.cos_sin = cos_sin


def _handle(stream):
    return None if stream is None else _stream(stream)


# ------------------------------------------------------------------ status-returning calls

def status_kv_append(cache, k, v, slots, rope=None, positions=None, q=None, q_out=None, status=None,
                     stream=None) -> int:
    return _binding.kv_append(cache._handle, k, v, slots, None if rope is None else rope._handle, positions, q,
                              q_out, status, _handle(stream))


def status_attn_decode(out, q, cache, block_table, seq_lens, max_len: int, scale: float, window: int = 0,
                       lse=None, workspace=None, status=None, stream=None) -> int:
    return _binding.attn_decode(out, q, cache._handle, block_table, seq_lens, max_len, scale, window, lse, workspace,
                                status, _handle(stream))


def status_attn_join(out, parts, lses, lse=None, stream=None) -> int:
    return _binding.attn_join(out, parts, lses, lse, _handle(stream))


# ------------------------------------------------------------------ raising calls (C names)

def detfold_kv_append(cache, k, v, slots, rope=None, positions=None, q=None, q_out=None, status=None,
                      stream=None) -> None:
    """Append k and v [tokens, kv_heads, head_dim] to the cache at slots [tokens]
    (int64, negative: padding), keys rotated by `rope` at positions [tokens] (int64);
    q [tokens, heads, head_dim] rotated into q_out (q itself: in place)."""
    rc = _binding.kv_append(cache._handle, k, v, slots, None if rope is None else rope._handle, positions, q, q_out,
                            status, None if stream is None else _stream(stream))
    if rc:
        _check(rc, "detfold_kv_append")


def detfold_attn_decode_workspace_bytes(cache, batch: int, q_heads: int, max_len: int) -> int:
    """Bytes of workspace that detfold_attn_decode needs for these sizes."""
    n = _binding.workspace_bytes(cache._handle, batch, q_heads, max_len)
    _check(n if n < 0 else 0, "detfold_attn_decode_workspace_bytes")
    return n


def detfold_attn_decode(out, q, cache, block_table, seq_lens, max_len: int, scale: float, window: int = 0,
                        lse=None, workspace=None, status=None, stream=None) -> None:
    """out [batch, heads, head_dim] = attention of the queries q over each
    sequence's cached tokens (the last `window` of them; 0: all). block_table
    [batch, cols] and seq_lens [batch] are int32; lse [batch, heads] is float32."""
    rc = _binding.attn_decode(out, q, cache._handle, block_table, seq_lens, max_len, scale, window, lse, workspace,
                              status, None if stream is None else _stream(stream))
    if rc:
        _check(rc, "detfold_attn_decode")


def detfold_attn_join(out, parts, lses, lse=None, stream=None) -> None:
    """out = the ranks' partial attentions `parts` (each of out's shape) joined by
    their `lses` (float32, out's shape without the last dimension), rank 0 first."""
    rc = _binding.attn_join(out, parts, lses, lse, None if stream is None else _stream(stream))
    if rc:
        _check(rc, "detfold_attn_join")


def detfold_attn_last_cuda_error() -> int:
    return lib.detfold_attn_last_cuda_error()
