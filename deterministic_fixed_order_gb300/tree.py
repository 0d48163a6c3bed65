"""Python binding of libdetfold_tree, a step with drafted tokens over the paged
key-value cache (``include/detfold_tree.h``).

Argument marshalling only, as in ``attention``: the functions keep the C names, a
negative status raises ``DetfoldError``, and the ``status_*`` variants return it
instead. ``stream`` may be None (torch's current stream), a ``torch.cuda.Stream``
or a raw handle. ``lib`` is the C ABI itself, through ctypes.
"""
from __future__ import annotations

import ctypes
import os

from . import DetfoldError, STATUS, _build, detfold_status_string
from .attention import _binding, _handle

__all__ = [
    "detfold_tree_plan", "detfold_attn_tree", "detfold_attn_tree_workspace_bytes", "detfold_kv_compact",
    "detfold_kv_copy_pages", "detfold_pages_step", "detfold_tree_last_cuda_error", "DETFOLD_TREE_MAX_NODES",
    "DETFOLD_PAGES_MAX_ROWS",
]

DETFOLD_TREE_MAX_NODES = 256
DETFOLD_PAGES_MAX_ROWS = 4096

TREE_LIB_PATH = _build.TREE_LIB
if not os.path.exists(TREE_LIB_PATH):
    raise ImportError(
        f"libdetfold_tree.so is not built ({TREE_LIB_PATH}); run "
        "`python -c 'import __graft_entry__ as g; g.build()'` first")

lib = ctypes.CDLL(TREE_LIB_PATH)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_F = ctypes.c_float

lib.detfold_tree_plan.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _INT, _I64, _INT, _INT, _P, _P]
lib.detfold_attn_tree_workspace_bytes.argtypes = [_P, _INT, _INT, _INT, _I64]
lib.detfold_attn_tree_workspace_bytes.restype = _I64
lib.detfold_attn_tree.argtypes = [_P, _I64, _I64, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _P, _INT,
                                  _INT, _INT, _I64, _F, _I64, _P, _I64, _P, _P]
lib.detfold_kv_compact.argtypes = [_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _INT, _P, _P]
lib.detfold_kv_copy_pages.argtypes = [_P, _P, _P, _P, _I64, _P, _P]
lib.detfold_pages_step.argtypes = [_P, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _INT, _INT,
                                   _INT, _P, _P]
lib.detfold_tree_last_cuda_error.argtypes = []
for _name in ("detfold_tree_plan", "detfold_attn_tree", "detfold_kv_compact", "detfold_kv_copy_pages",
              "detfold_pages_step", "detfold_tree_last_cuda_error"):
    getattr(lib, _name).restype = _INT


class TreeError(DetfoldError):
    """A failed CUDA call of this library (its error value is kept apart from the other libraries')."""

    def __init__(self, status: int, where: str):
        RuntimeError.__init__(self, f"{where}: status {status}: {detfold_status_string(status)} "
                                    f"(cudaError {lib.detfold_tree_last_cuda_error()})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != 0:
        if status == STATUS["DETFOLD_ERR_CUDA"]:
            raise TreeError(status, where)
        raise DetfoldError(status, where)


# ------------------------------------------------------------------ status-returning calls

def status_tree_plan(mask, parents, seq_lens, block_table=None, page_size: int = 1, num_pages: int = 0,
                     node_counts=None, positions=None, slots=None, status=None, stream=None) -> int:
    return _binding.tree_plan(mask, parents, seq_lens, node_counts, block_table, page_size, num_pages, positions,
                              slots, status, _handle(stream))


def status_attn_tree(out, q, cache, block_table, seq_lens, mask, max_len: int, scale: float, node_counts=None,
                     window: int = 0, lse=None, workspace=None, status=None, stream=None) -> int:
    return _binding.attn_tree(out, q, cache._handle, block_table, seq_lens, mask, max_len, scale, node_counts, window,
                              lse, workspace, status, _handle(stream))


def status_kv_compact(cache, block_table, seq_lens, path, path_lens, status=None, stream=None) -> int:
    return _binding.kv_compact(cache._handle, block_table, seq_lens, path, path_lens, status, _handle(stream))


def status_kv_copy_pages(cache, src, dst, rows=None, status=None, stream=None) -> int:
    return _binding.kv_copy_pages(cache._handle, src, dst, rows, status, _handle(stream))


def status_pages_step(refs_out, table_out, lens_out, copy_src, copy_dst, copy_rows, refs, table, lens, origin, keep,
                      want, page_size: int, status=None, stream=None) -> int:
    return _binding.pages_step(refs_out, table_out, lens_out, copy_src, copy_dst, copy_rows, refs, table, lens, origin,
                               keep, want, page_size, status, _handle(stream))


# ------------------------------------------------------------------ raising calls (C names)

def detfold_tree_plan(mask, parents, seq_lens, block_table=None, page_size: int = 1, num_pages: int = 0,
                      node_counts=None, positions=None, slots=None, status=None, stream=None) -> None:
    """Ancestor bits mask [batch, nodes, words] (int64, a word for 64 nodes) of trees given by
    parents [batch, nodes] (int32, -1: follows the committed tokens); positions and slots
    [batch, nodes] (int64) for detfold_kv_append. seq_lens and node_counts [batch] are int32."""
    _check(status_tree_plan(mask, parents, seq_lens, block_table, page_size, num_pages, node_counts, positions, slots,
                            status, stream), "detfold_tree_plan")


def detfold_attn_tree_workspace_bytes(cache, batch: int, nodes: int, q_heads: int, max_len: int) -> int:
    """Bytes of workspace that detfold_attn_tree needs for these sizes."""
    n = _binding.tree_workspace_bytes(cache._handle, batch, nodes, q_heads, max_len)
    _check(n if n < 0 else 0, "detfold_attn_tree_workspace_bytes")
    return n


def detfold_attn_tree(out, q, cache, block_table, seq_lens, mask, max_len: int, scale: float, node_counts=None,
                      window: int = 0, lse=None, workspace=None, status=None, stream=None) -> None:
    """out [batch, nodes, heads, head_dim] = attention of the queries q of each tree's nodes over
    the committed tokens (with a window, the last ones before the node) and the drafted
    ones that the node's mask names. lse [batch, nodes, heads] is float32."""
    _check(status_attn_tree(out, q, cache, block_table, seq_lens, mask, max_len, scale, node_counts, window, lse,
                            workspace, status, stream), "detfold_attn_tree")


def detfold_kv_compact(cache, block_table, seq_lens, path, path_lens, status=None, stream=None) -> None:
    """Rows of the accepted nodes path [batch, max_path] (int32, ascending; the first
    path_lens [batch] of them) move to the end of the committed tokens seq_lens [batch]."""
    _check(status_kv_compact(cache, block_table, seq_lens, path, path_lens, status, stream), "detfold_kv_compact")


def detfold_kv_copy_pages(cache, src, dst, rows=None, status=None, stream=None) -> None:
    """Pages src [n] of the cache (int32; the first rows [n] rows of each) to pages dst [n]."""
    _check(status_kv_copy_pages(cache, src, dst, rows, status, stream), "detfold_kv_copy_pages")


def detfold_pages_step(refs_out, table_out, lens_out, copy_src, copy_dst, copy_rows, refs, table, lens, origin, keep,
                       want, page_size: int, status=None, stream=None) -> None:
    """One step of a pool's bookkeeping (include/detfold_tree.h): new rows keep the first `keep`
    tokens of the rows `origin` of the block table and get room for `want`. All int32;
    copy_src, copy_dst and copy_rows are what detfold_kv_copy_pages has to copy next."""
    _check(status_pages_step(refs_out, table_out, lens_out, copy_src, copy_dst, copy_rows, refs, table, lens, origin,
                             keep, want, page_size, status, stream), "detfold_pages_step")


def detfold_tree_last_cuda_error() -> int:
    return lib.detfold_tree_last_cuda_error()
