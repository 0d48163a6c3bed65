"""The C boundary of the library of drafted steps on the CPU: its symbols, its constants and
the refusals of its argument checks. No call here reaches a kernel launch."""
import ctypes
import glob
import os
import re
import subprocess

import pytest

from test_attn_abi import A, cache, no_gpu_only

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "detfold_tree.h")
TREE = os.path.join(ROOT, "deterministic_fixed_order_gb300", "csrc", "tree")

EXPORTED_API = {"detfold_tree_plan", "detfold_attn_tree", "detfold_attn_tree_workspace_bytes", "detfold_kv_compact",
                "detfold_kv_copy_pages", "detfold_pages_step", "detfold_tree_last_cuda_error"}


@pytest.fixture(scope="module")
def df():
    import deterministic_fixed_order_gb300 as m
    return m


def test_header_and_library_name_the_same_calls(df):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert set(re.findall(r"\b(detfold_\w+)\s*\(", text)) == EXPORTED_API
    out = subprocess.run(["nm", "-D", "--defined-only", df.tree.TREE_LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert {line.split()[-1] for line in out.splitlines() if line.strip()} == EXPORTED_API


def test_header_compiles_as_c():
    src = '#include "detfold_tree.h"\nint main(void){return DETFOLD_TREE_WORDS(65) - 2;}\n'
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-x", "c", "-", "-o",
                        os.devnull], input=src, text=True, capture_output=True)
    assert r.returncode == 0, r.stderr


def test_binding_constants_match_the_header(df):
    defs = dict(re.findall(r"^#define (DETFOLD_\w+) (.+)$", open(HEADER).read(), re.M))
    for name in ("DETFOLD_TREE_MAX_NODES", "DETFOLD_PAGES_MAX_ROWS"):
        assert getattr(df.tree, name) == int(defs[name]), name


def test_names_of_the_package(df):
    for name in EXPORTED_API - {"detfold_tree_last_cuda_error"}:
        assert getattr(df, name) is getattr(df.tree, name)


def test_kernels_wait_before_they_read():
    """Every kernel here may start before the launch ahead of it has ended: it waits once, outside
    every branch, and reads nothing before."""
    for path in glob.glob(os.path.join(TREE, "*.cu*")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\benter_grid\(\);", text):
            before = text[:m.start()]
            start = max(x.start() for x in re.finditer(r"__global__|static __device__", before))
            head = before[start:]
            assert head.count("{") - head.count("}") == 1, path
            assert not re.search(r"\bp\.(lens|counts|parents|path|refs|src|table)\[|tree_seq_of", head), path
        assert len(re.findall(r"__global__", text)) <= len(re.findall(r"\benter_grid\(\);", text)), path


# ------------------------------------------------------------------ refusals

def tree_args(df, **kw):
    d = kw.pop("cache_kw", {})
    a = dict(out=A + (2 << 24), out_bs=8 * 256, out_ns=256, out_hs=64, lse=0, q=A + (3 << 24), q_bs=8 * 256, q_ns=256,
             q_hs=64, cache=ctypes.byref(cache(df, **d)), table=A + (4 << 24), ts=4, tc=4, lens=A + (5 << 24), counts=0,
             mask=A + (6 << 24), batch=2, nodes=8, heads=4, max_len=64, scale=1.0, window=0, ws=A + (7 << 24),
             ws_bytes=1 << 22, status=0, stream=0)
    a.update(kw)
    return list(a.values())


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(out=0), -1), (dict(q=0), -1), (dict(lens=0), -1), (dict(mask=0), -1), (dict(table=0), -1), (dict(cache=None), -1),
    (dict(cache_kw=dict(k=0)), -1), (dict(nodes=257), -8), (dict(nodes=-1), -8), (dict(batch=-1), -8), (dict(heads=3), -8),
    (dict(heads=0), -8), (dict(window=7), -8), (dict(window=-1), -8), (dict(max_len=65), -3), (dict(max_len=-1), -3),
    (dict(max_len=(1 << 30) + 1, tc=1 << 40), -3), (dict(cache_kw=dict(head_dim=264)), -8), (dict(cache_kw=dict(dtype=3)), -8),
    (dict(cache_kw=dict(head_dim=60)), -4), (dict(cache_kw=dict(k=A + 8)), -4), (dict(cache_kw=dict(token_stride=132)), -4),
    (dict(out=A + (2 << 24) + 1), -4), (dict(mask=A + 4), -4), (dict(counts=A + 2), -4), (dict(status=A + 2), -4),
    (dict(out_hs=63), -8), (dict(out_ns=63), -8), (dict(out_bs=63), -8), (dict(q_bs=-1), -8), (dict(ts=-1), -8),
    (dict(out=A + (3 << 24)), -5), (dict(out=A), -5), (dict(lse=A + (3 << 24)), -5), (dict(lse=A + (6 << 24)), -5),
    (dict(max_len=100000, tc=100000, ws=0), -6), (dict(max_len=100000, tc=100000, ws_bytes=100), -6),
    (dict(max_len=100000, tc=100000, ws=A + 8 + (7 << 24), ws_bytes=1 << 40), -6),
    (dict(max_len=100000, tc=100000, ws=A + (3 << 24), ws_bytes=1 << 40), -5),
    (dict(batch=1 << 20, nodes=256, out_bs=1 << 20), -5),  # 2^30 rows, the most that there may be
    (dict(batch=1 << 20, nodes=256, heads=8, out_bs=1 << 20), -8), (dict(out_bs=1 << 50), -8),
])
def test_attn_tree_refusals(df, kw, status):
    assert df.tree.lib.detfold_attn_tree(*tree_args(df, **kw)) == status


@no_gpu_only
def test_calls_without_rows(df):
    lib = df.tree.lib
    assert lib.detfold_attn_tree(*tree_args(df, batch=0, out=0, q=0, lens=0, mask=0, ws=0, table=0)) == 0
    assert lib.detfold_attn_tree(*tree_args(df, nodes=0, out=0, q=0, lens=0, mask=0, ws=0)) == 0
    c = ctypes.byref(cache(df))
    assert lib.detfold_kv_compact(c, 0, 0, 0, 0, 0, 0, 0, 0, 3, 0, 0) == 0
    assert lib.detfold_kv_compact(c, 0, 0, 0, 0, 0, 0, 0, 3, 0, 0, 0) == 0
    assert lib.detfold_kv_copy_pages(c, 0, 0, 0, 0, 0, 0) == 0
    assert lib.detfold_tree_plan(0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 1, 0, 5, 0, 0) == 0
    assert lib.detfold_tree_plan(0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 1, 5, 0, 0, 0) == 0


B, C, D, E, F = (A + (i << 24) for i in range(2, 7))


@no_gpu_only
@pytest.mark.parametrize("change,status", [
    ({0: 0}, -1), ({3: 0}, -1), ({4: 0}, -1), ({6: 0}, -1), ({11: -1}, -8), ({12: 257}, -8), ({9: 0}, -8), ({10: -1}, -8),
    ({7: -1}, -8), ({0: B + 4}, -4), ({1: C + 4}, -4), ({3: E + 2}, -4), ({1: B}, -5), ({0: E}, -5), ({2: F}, -5), ({13: 2}, -4),
    ({11: (1 << 20) + 1}, -8),
])
def test_plan_refusals(df, change, status):
    a = [B, C, D, E, E + 4096, 0, F, 4, 4, 16, 9, 2, 8, 0, 0]
    for i, x in change.items():
        a[i] = x
    assert df.tree.lib.detfold_tree_plan(*a) == status


@no_gpu_only
@pytest.mark.parametrize("change,kw,status", [
    ({1: 0}, {}, -1), ({4: 0}, {}, -1), ({5: 0}, {}, -1), ({7: 0}, {}, -1), ({8: -1}, {}, -8), ({9: 257}, {}, -8), ({2: -1}, {}, -8),
    ({6: -1}, {}, -8), ({5: C + 1}, {}, -4), ({10: 1}, {}, -4), ({5: A}, {}, -5), ({1: A + 64}, {}, -5), ({}, dict(k=0), -1),
    ({}, dict(k=A + 1), -4), ({}, dict(head_stride=63), -8), ({}, dict(token_stride=63), -8), ({}, dict(page_stride=63), -8),
    ({}, dict(num_pages=1 << 31), -8), ({}, dict(page_size=1 << 20, kv_heads=1 << 8, head_dim=8, head_stride=8, token_stride=2048,
                                              page_stride=1 << 31, k=1 << 50), -8),
])
def test_compact_refusals(df, change, kw, status):
    a = [ctypes.byref(cache(df, **kw)), B, 4, 4, C, D, 8, E, 2, 8, 0, 0]
    for i, x in change.items():
        a[i] = x
    assert df.tree.lib.detfold_kv_compact(*a) == status


@no_gpu_only
@pytest.mark.parametrize("change,kw,status", [
    ({1: 0}, {}, -1), ({2: 0}, {}, -1), ({4: -1}, {}, -3), ({4: (1 << 30) + 1}, {}, -3), ({1: B + 2}, {}, -4), ({3: D + 1}, {}, -4),
    ({2: A}, {}, -5), ({5: 3}, {}, -4), ({}, dict(v=0), -1), ({}, dict(head_stride=63), -8),
])
def test_copy_refusals(df, change, kw, status):
    a = [ctypes.byref(cache(df, **kw)), B, C, D, 5, 0, 0]
    for i, x in change.items():
        a[i] = x
    assert df.tree.lib.detfold_kv_copy_pages(*a) == status


@no_gpu_only
@pytest.mark.parametrize("change,status", [
    ({0: 0}, -1), ({1: 0}, -1), ({3: 0}, -1), ({4: 0}, -1), ({7: 0}, -1), ({8: 0}, -1), ({10: 0}, -1), ({11: 0}, -1), ({13: 0}, -1),
    ({14: 0}, -8), ({14: (1 << 30) + 1}, -8), ({15: -1}, -8), ({15: (1 << 20) + 1}, -8), ({16: 0}, -8), ({17: 4097}, -8), ({17: -1}, -8),
    ({18: 4097}, -8), ({2: 3}, -8), ({2: -1}, -8), ({9: -1}, -8), ({0: B + 2}, -4), ({19: 2}, -4), ({1: D}, -5), ({0: D}, -5),
    ({3: E + 256}, -5), ({7: B + 4}, -5), ({0: E}, -5),
])
def test_pages_refusals(df, change, status):
    a = [B, C, 4, E + 1024, E + 2048, E + 3 * 1024, E + 4096, B, D, 4, E, E + 64, E + 128, E + 256, 100, 4, 16, 3, 5, 0, 0]
    for i, x in change.items():
        a[i] = x
    assert df.tree.lib.detfold_pages_step(*a) == status


def test_workspace_only_grows(df):
    """No sizes need less for a larger max_len, a larger batch or larger trees; invalid ones are refused."""
    need = df.tree.lib.detfold_attn_tree_workspace_bytes
    for dtype, d in ((0, 64), (1, 64), (1, 128), (2, 192), (2, 256), (0, 256)):
        for kv, group in ((1, 1), (8, 4), (2, 16), (40, 1), (1, 130)):
            c = cache(df, dtype=dtype, head_dim=d, kv_heads=kv)
            for nodes in (1, 7, 32, 33, 256):
                sizes = [need(ctypes.byref(c), 3, nodes, kv * group, n) for n in (0, 1, 64, 257, 1000, 1024, 1025, 5000, 40000, 1 << 30)]
                assert sizes == sorted(sizes) and sizes[0] >= 0
                assert need(ctypes.byref(c), 4, nodes, kv * group, 5000) >= sizes[7]
    c = cache(df)
    for bad in ((-1, 8, 4, 10), (1, 257, 4, 10), (1, 8, 3, 10), (1, 8, 4, -1), (1, 8, 4, (1 << 30) + 1), (1, 8, 0, 10)):
        assert need(ctypes.byref(c), *bad) < 0
    assert need(None, 1, 8, 4, 10) == -1
