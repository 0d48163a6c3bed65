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


def _type_code(dtype, what: str) -> int:
    if not _TYPES:
        torch = _t()
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


def _want(x, dtype, device: int, dims: int, what: str):
    """x as a CUDA tensor of this type, device and rank, its last dimension contiguous."""
    if x.dtype is not dtype or x.get_device() != device:
        raise TypeError(f"{what}: expected a {dtype} tensor on cuda:{device}, got {x.dtype} on {x.device}")
    if x.dim() != dims:
        raise ValueError(f"{what}: expected {dims} dimensions, got shape {tuple(x.shape)}")
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return x


def _flat(x, dtype, device: int, count: int, what: str) -> int:
    """Address of a contiguous CUDA tensor of this type with `count` elements."""
    if x.dtype is not dtype or x.get_device() != device:
        raise TypeError(f"{what}: expected a {dtype} tensor on cuda:{device}, got {x.dtype} on {x.device}")
    if not x.is_contiguous() or x.numel() != count:
        raise ValueError(f"{what}: expected {count} contiguous elements, got shape {tuple(x.shape)}")
    return x.data_ptr()


def _status_word(status, device: int) -> int:
    if status is None:
        return 0
    torch = _t()
    if status.dtype is not torch.int32 or status.get_device() != device or status.numel() < 1:
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
        _want(k, k.dtype, self.device, 4, "k")
        _want(v, k.dtype, self.device, 4, "v")
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
        torch = _t()
        if cos_sin.dtype is not torch.float32 or not cos_sin.is_cuda:
            raise TypeError(f"cos_sin: expected a CUDA float32 tensor, got {cos_sin.device} {cos_sin.dtype}")
        if cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin: expected a contiguous [positions, rot_dim] tensor")
        self.cos_sin, self.device = cos_sin, cos_sin.get_device()
        self._desc = _Rope(cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], 1 if interleaved else 0)
        self._ptr = ctypes.addressof(self._desc)


# ------------------------------------------------------------------ status-returning calls

def status_kv_append(cache, k, v, slots, rope=None, positions=None, q=None, q_out=None, status=None,
                     stream=None) -> int:
    torch = _t()
    device, dtype = cache.device, cache.dtype
    _want(k, dtype, device, 3, "k")
    _want(v, dtype, device, 3, "v")
    tokens, heads, width = k.shape
    if heads != cache.kv_heads or width != cache.head_dim or v.shape != k.shape:
        raise ValueError(f"k and v: expected [tokens, {cache.kv_heads}, {cache.head_dim}], got "
                         f"{tuple(k.shape)} and {tuple(v.shape)}")
    slot_ptr = _flat(slots, torch.int64, device, tokens, "slots")
    rope_ptr = pos_ptr = 0
    if rope is not None:
        if rope.device != device:
            raise TypeError("rope: on another device than the cache")
        if positions is None:
            raise ValueError("positions: needed with rope")
        rope_ptr, pos_ptr = rope._ptr, _flat(positions, torch.int64, device, tokens, "positions")
    ks, vs = k.stride(), v.stride()
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        return lib.detfold_kv_append(cache._ptr, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                                     slot_ptr, tokens, rope_ptr, pos_ptr, 0, 0, 0, 0, 0, 0, 0,
                                     _status_word(status, device), _stream(stream))
    _want(q, dtype, device, 3, "q")
    if q_out is None:
        raise ValueError("q_out: needed with q")
    _want(q_out, dtype, device, 3, "q_out")
    if q.shape[0] != tokens or q.shape[2] != width or q_out.shape != q.shape:
        raise ValueError(f"q and q_out: expected [{tokens}, heads, {width}], got {tuple(q.shape)} and "
                         f"{tuple(q_out.shape)}")
    qs, os_ = q.stride(), q_out.stride()
    return lib.detfold_kv_append(cache._ptr, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], slot_ptr,
                                 tokens, rope_ptr, pos_ptr, q_out.data_ptr(), os_[0], os_[1], q.data_ptr(),
                                 qs[0], qs[1], q.shape[1], _status_word(status, device), _stream(stream))


def status_attn_decode(out, q, cache, block_table, seq_lens, max_len: int, scale: float, window: int = 0,
                       lse=None, workspace=None, status=None, stream=None) -> int:
    torch = _t()
    device, dtype = cache.device, cache.dtype
    _want(q, dtype, device, 3, "q")
    _want(out, dtype, device, 3, "out")
    batch, heads, width = q.shape
    if width != cache.head_dim or out.shape != q.shape:
        raise ValueError(f"q and out: expected [batch, heads, {cache.head_dim}], got {tuple(q.shape)} and "
                         f"{tuple(out.shape)}")
    _want(block_table, torch.int32, device, 2, "block_table")
    rows, cols = block_table.shape
    if rows != batch:
        raise ValueError(f"block_table: expected {batch} rows, got {rows}")
    lens_ptr = _flat(seq_lens, torch.int32, device, batch, "seq_lens")
    lse_ptr = 0 if lse is None else _flat(lse, torch.float32, device, batch * heads, "lse")
    ws_ptr = ws_bytes = 0
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on cuda:{device}")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    os_, qs = out.stride(), q.stride()
    return lib.detfold_attn_decode(out.data_ptr(), os_[0], os_[1], lse_ptr, q.data_ptr(), qs[0], qs[1],
                                   cache._ptr, block_table.data_ptr(), block_table.stride(0), cols, lens_ptr,
                                   batch, heads, max_len, scale, window, ws_ptr, ws_bytes,
                                   _status_word(status, device), _stream(stream))


def status_attn_join(out, parts, lses, lse=None, stream=None) -> int:
    torch = _t()
    world, device = len(parts), out.get_device()
    if len(lses) != world:
        raise ValueError(f"{world} parts, {len(lses)} lses")
    code = _type_code(out.dtype, "out")
    count, width = out.numel(), out.shape[-1] if out.dim() else 0
    rows = count // width if width else 0
    if not out.is_cuda:
        raise TypeError(f"out: expected a CUDA tensor, got {out.device}")
    table = _pointers(world)
    part_ptrs = table(*[_flat(x, out.dtype, device, count, "parts") for x in parts])
    lse_ptrs = table(*[_flat(x, torch.float32, device, rows, "lses") for x in lses])
    return lib.detfold_attn_join(_flat(out, out.dtype, device, count, "out"),
                                 0 if lse is None else _flat(lse, torch.float32, device, rows, "lse"),
                                 part_ptrs, lse_ptrs, world, rows, width, code, _stream(stream))


_POINTERS = {}  # ctypes pointer-array types by length


def _pointers(n: int):
    got = _POINTERS.get(n)
    if got is None:
        got = _POINTERS.setdefault(n, ctypes.c_void_p * n)
    return got


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
