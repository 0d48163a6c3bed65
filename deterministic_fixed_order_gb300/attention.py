"""Python binding of libdetfold_attn, the decode step's attention over a paged
key-value cache (``include/detfold_attn.h``).

Argument marshalling only, as in the package itself: the functions keep the C
names, check the tensors that they are given (device, type, shape, strides) and
pass addresses on; the library checks the rest. ``stream`` may be None (torch's
current stream), a ``torch.cuda.Stream`` or a raw handle. A negative status
raises ``DetfoldError``; the ``status_*`` variants return it instead.

``PagedCache`` and ``Rope`` hold what a program keeps between calls: the cache
and the table of rotations, described once. They keep their tensors alive.
"""
from __future__ import annotations

import ctypes
import os

from . import DetfoldError, STATUS, _build, _stream, _t, detfold_status_string

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

_TYPES = {}  # torch types, filled on first use
_F32 = _I32 = _I64T = None
_POINTERS = {}  # ctypes pointer-array types by length


def _type_code(dtype, what: str) -> int:
    global _F32, _I32, _I64T
    if not _TYPES:
        torch = _t()
        _F32, _I32, _I64T = torch.float32, torch.int32, torch.int64
        _TYPES.update({torch.float32: DETFOLD_F32, torch.bfloat16: DETFOLD_BF16, torch.float16: DETFOLD_F16})
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError(f"{what}: expected float32, bfloat16 or float16, got {dtype}")
    return code


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


# The checks below run on every call and are written for that: the accepted case
# asks each tensor for as little as it can, the messages are made on refusal.

def _refuse(x, dtype, device: int, shape, what: str):
    """Raises for a tensor that is not of this type, device and shape (None: any
    length), or whose last dimension is not contiguous."""
    if not hasattr(x, "get_device"):
        raise TypeError(f"{what}: expected a tensor, got {type(x).__name__}")
    if x.dtype is not dtype or x.get_device() != device:
        raise TypeError(f"{what}: expected a {dtype} tensor on cuda:{device}, got {x.dtype} on {x.device}")
    text = "[" + ", ".join("any" if n is None else str(n) for n in shape) + "]"
    if x.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, x.shape)):
        raise ValueError(f"{what}: expected shape {text}, got {tuple(x.shape)}")
    raise ValueError(f"{what}: strides {x.stride()} of shape {text}: the last dimension must be contiguous")


def _rows(x, dtype, device: int, shape, what: str):
    """(address, first stride, second stride) of [shape[0], shape[1], shape[2]] with a contiguous last dimension."""
    s = x.stride()
    if x.dtype is not dtype or x.get_device() != device or x.shape != shape or (s[2] != 1 and shape[2] > 1):
        _refuse(x, dtype, device, shape, what)
    return x.data_ptr(), s[0], s[1]


def _flat(x, dtype, device: int, count: int, what: str) -> int:
    """Address of a contiguous CUDA tensor of this type with `count` elements."""
    if x.dtype is not dtype or x.get_device() != device:
        _refuse(x, dtype, device, (count,), what)
    if not x.is_contiguous() or x.numel() != count:
        raise ValueError(f"{what}: expected {count} contiguous elements, got shape {tuple(x.shape)}, strides "
                         f"{x.stride()}")
    return x.data_ptr()


def _status_word(status, device: int) -> int:
    if status.dtype is not _I32 or status.get_device() != device or status.numel() < 1:
        raise TypeError("status: expected a CUDA int32 tensor")
    return status.data_ptr()


class PagedCache:
    """A paged cache: k and v of shape [pages, page_size, kv_heads, head_dim] with
    the same strides, any order of the first three dimensions (a view of a
    cache that is stored head by head, or of one buffer that holds both)."""

    def __init__(self, k, v):
        code = _type_code(k.dtype, "k")
        if not k.is_cuda:
            raise TypeError(f"k: expected a CUDA tensor, got {k.device}")
        self.device, self.dtype = k.get_device(), k.dtype
        for x, what in ((k, "k"), (v, "v")):
            if x.dtype is not k.dtype or x.get_device() != self.device or x.dim() != 4 or (
                    x.stride(3) != 1 and x.shape[3] > 1):
                _refuse(x, k.dtype, self.device, (None,) * 4, what)
        if k.shape != v.shape or k.stride() != v.stride():
            raise ValueError(f"k and v differ: shapes {tuple(k.shape)} and {tuple(v.shape)}, strides "
                             f"{k.stride()} and {v.stride()}")
        pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.k, self.v = k, v
        s = k.stride()
        self._desc = _Cache(k.data_ptr(), v.data_ptr(), pages, s[0], s[1], s[2], code, self.page_size,
                            self.kv_heads, self.head_dim)
        self._ptr = ctypes.addressof(self._desc)


class Rope:
    """A table of rotations: cos_sin [positions, rot_dim] float32, cosines then
    sines. Pairs are elements (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved."""

    def __init__(self, cos_sin, interleaved: bool = False):
        if cos_sin.dtype is not _t().float32 or not cos_sin.is_cuda:
            raise TypeError(f"cos_sin: expected a CUDA float32 tensor, got {cos_sin.device} {cos_sin.dtype}")
        if cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin: expected a contiguous [positions, rot_dim] tensor")
        self.cos_sin, self.device = cos_sin, cos_sin.get_device()
        self._desc = _Rope(cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], 1 if interleaved else 0)
        self._ptr = ctypes.addressof(self._desc)


# ------------------------------------------------------------------ status-returning calls

def status_kv_append(cache, k, v, slots, rope=None, positions=None, q=None, q_out=None, status=None,
                     stream=None) -> int:
    device, dtype = cache.device, cache.dtype
    shape = k.shape
    tokens = shape[0] if len(shape) == 3 else 0
    if len(shape) != 3 or shape[1] != cache.kv_heads or shape[2] != cache.head_dim:
        _refuse(k, dtype, device, (None, cache.kv_heads, cache.head_dim), "k")
    k_ptr, k_ts, k_hs = _rows(k, dtype, device, shape, "k")
    v_ptr, v_ts, v_hs = _rows(v, dtype, device, shape, "v")
    slot_ptr = _flat(slots, _I64T, device, tokens, "slots")
    rope_ptr = pos_ptr = 0
    if rope is not None:
        if rope.device != device:
            raise TypeError("rope: on another device than the cache")
        if positions is None:
            raise ValueError("positions: needed with rope")
        rope_ptr, pos_ptr = rope._ptr, _flat(positions, _I64T, device, tokens, "positions")
    q_ptr = q_ts = q_hs = o_ptr = o_ts = o_hs = heads = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q_out: needed with q")
        shape = q.shape
        if len(shape) != 3 or shape[0] != tokens or shape[2] != cache.head_dim:
            _refuse(q, dtype, device, (tokens, None, cache.head_dim), "q")
        heads = shape[1]
        q_ptr, q_ts, q_hs = _rows(q, dtype, device, shape, "q")
        o_ptr, o_ts, o_hs = _rows(q_out, dtype, device, shape, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    return lib.detfold_kv_append(cache._ptr, k_ptr, k_ts, k_hs, v_ptr, v_ts, v_hs, slot_ptr, tokens, rope_ptr, pos_ptr,
                                 o_ptr, o_ts, o_hs, q_ptr, q_ts, q_hs, heads,
                                 0 if status is None else _status_word(status, device), _stream(stream))


def status_attn_decode(out, q, cache, block_table, seq_lens, max_len: int, scale: float, window: int = 0,
                       lse=None, workspace=None, status=None, stream=None) -> int:
    device, dtype = cache.device, cache.dtype
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim:
        _refuse(q, dtype, device, (None, None, cache.head_dim), "q")
    batch, heads, _ = shape
    q_ptr, q_bs, q_hs = _rows(q, dtype, device, shape, "q")
    o_ptr, o_bs, o_hs = _rows(out, dtype, device, shape, "out")
    table, ts = block_table.shape, block_table.stride()
    if block_table.dtype is not _I32 or block_table.get_device() != device or len(table) != 2 or (
            table[0] != batch or (ts[1] != 1 and table[1] > 1)):
        _refuse(block_table, _I32, device, (batch, None), "block_table")
    lens_ptr = _flat(seq_lens, _I32, device, batch, "seq_lens")
    ws_ptr = ws_bytes = 0
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on cuda:{device}")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.nbytes
    return lib.detfold_attn_decode(o_ptr, o_bs, o_hs, 0 if lse is None else _flat(lse, _F32, device, batch * heads, "lse"),
                                   q_ptr, q_bs, q_hs, cache._ptr, block_table.data_ptr(), ts[0], table[1], lens_ptr,
                                   batch, heads, max_len, scale, window, ws_ptr, ws_bytes,
                                   0 if status is None else _status_word(status, device), _stream(stream))


def status_attn_join(out, parts, lses, lse=None, stream=None) -> int:
    world, device, dtype = len(parts), out.get_device(), out.dtype
    if len(lses) != world:
        raise ValueError(f"{world} parts, {len(lses)} lses")
    code = _type_code(dtype, "out")
    if device < 0:
        raise TypeError(f"out: expected a CUDA tensor, got {out.device}")
    count, shape = out.numel(), out.shape
    width = shape[-1] if shape else 0
    rows = count // width if width else 0
    table = _POINTERS.get(world) or _POINTERS.setdefault(world, ctypes.c_void_p * world)
    part_ptrs = table(*[_flat(x, dtype, device, count, "parts") for x in parts])
    lse_ptrs = table(*[_flat(x, _F32, device, rows, "lses") for x in lses])
    return lib.detfold_attn_join(_flat(out, dtype, device, count, "out"),
                                 0 if lse is None else _flat(lse, _F32, device, rows, "lse"),
                                 part_ptrs, lse_ptrs, world, rows, width, code, _stream(stream))


# ------------------------------------------------------------------ raising calls (C names)

def detfold_kv_append(cache, k, v, slots, rope=None, positions=None, q=None, q_out=None, status=None,
                      stream=None) -> None:
    """Append k and v [tokens, kv_heads, head_dim] to the cache at slots [tokens]
    (int64, negative: padding), keys rotated by `rope` at positions [tokens] (int64);
    q [tokens, heads, head_dim] rotated into q_out (q itself: in place)."""
    _check(status_kv_append(cache, k, v, slots, rope, positions, q, q_out, status, stream),
           "detfold_kv_append")


def detfold_attn_decode_workspace_bytes(cache, batch: int, q_heads: int, max_len: int) -> int:
    """Bytes of workspace that detfold_attn_decode needs for these sizes."""
    n = lib.detfold_attn_decode_workspace_bytes(cache._ptr, batch, q_heads, max_len)
    _check(n if n < 0 else 0, "detfold_attn_decode_workspace_bytes")
    return n


def detfold_attn_decode(out, q, cache, block_table, seq_lens, max_len: int, scale: float, window: int = 0,
                        lse=None, workspace=None, status=None, stream=None) -> None:
    """out [batch, heads, head_dim] = attention of the queries q over each
    sequence's cached tokens (the last `window` of them; 0: all). block_table
    [batch, cols] and seq_lens [batch] are int32; lse [batch, heads] is float32."""
    _check(status_attn_decode(out, q, cache, block_table, seq_lens, max_len, scale, window, lse, workspace,
                              status, stream), "detfold_attn_decode")


def detfold_attn_join(out, parts, lses, lse=None, stream=None) -> None:
    """out = the ranks' partial attentions `parts` (each of out's shape) joined by
    their `lses` (float32, out's shape without the last dimension), rank 0 first."""
    _check(status_attn_join(out, parts, lses, lse, stream), "detfold_attn_join")


def detfold_attn_last_cuda_error() -> int:
    return lib.detfold_attn_last_cuda_error()
