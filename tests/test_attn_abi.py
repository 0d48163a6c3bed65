"""The attention library's C boundary on the CPU: its symbols, its constants and
the refusals of its argument checks. No call here reaches a kernel launch."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "detfold_attn.h")

EXPORTED_API = {"detfold_kv_append", "detfold_attn_decode", "detfold_attn_decode_workspace_bytes",
                "detfold_attn_join", "detfold_attn_last_cuda_error"}


@pytest.fixture(scope="module")
def df():
    import deterministic_fixed_order_gb300 as m
    return m


def test_header_and_library_name_the_same_calls(df):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert set(re.findall(r"\b(detfold_\w+)\s*\(", text)) == EXPORTED_API
    out = subprocess.run(["nm", "-D", "--defined-only", df.attention.ATTN_LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert {line.split()[-1] for line in out.splitlines() if line.strip()} == EXPORTED_API


def test_header_compiles_as_c():
    src = '#include "detfold_attn.h"\nint main(void){detfold_kv_cache c; c.k = 0; return c.k != 0;}\n'
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-x", "c", "-", "-o",
                        os.devnull], input=src, text=True, capture_output=True)
    assert r.returncode == 0, r.stderr


def test_binding_constants_match_the_header(df):
    defs = dict(re.findall(r"^#define (DETFOLD_\w+) (.+)$", open(HEADER).read(), re.M))
    assert df.attention.DETFOLD_ATTN_MAX_LEN == 1 << 30 and "<< 30" in defs["DETFOLD_ATTN_MAX_LEN"]
    assert df.attention.DETFOLD_ATTN_MAX_COUNT == 1 << 20 and "<< 20" in defs["DETFOLD_ATTN_MAX_COUNT"]
    for name in ("DETFOLD_F32", "DETFOLD_BF16", "DETFOLD_F16", "DETFOLD_ATTN_MAX_HEAD_DIM"):
        assert getattr(df.attention, name) == int(defs[name]), name


def test_binding_structures_match_the_header(df):
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "detfold_attn.h"\nint main(void){'
           'printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(detfold_kv_cache), offsetof(detfold_kv_cache, head_stride),'
           'offsetof(detfold_kv_cache, head_dim), sizeof(detfold_rope), offsetof(detfold_rope, positions),'
           'offsetof(detfold_rope, interleaved)); return 0;}\n')
    import tempfile
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "layout")
        subprocess.run(["gcc", "-I", os.path.dirname(HEADER), "-x", "c", "-", "-o", exe], input=src, text=True, check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    c, r = df.attention._Cache, df.attention._Rope
    assert got == [ctypes.sizeof(c), c.head_stride.offset, c.head_dim.offset, ctypes.sizeof(r), r.positions.offset,
                   r.interleaved.offset]


# Fake device addresses, passed only where no GPU exists.
A = 1 << 32


def _has_gpu():
    try:
        import torch
        return torch.cuda.is_available() or os.path.exists("/dev/nvidia0")
    except Exception:
        return True


no_gpu_only = pytest.mark.skipif(_has_gpu(), reason="fake device addresses only where no GPU exists")


def cache(df, **kw):
    a = dict(k=A, v=A + (1 << 24), num_pages=4, page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64, dtype=1,
             page_size=16, kv_heads=2, head_dim=64)
    a.update(kw)
    return df.attention._Cache(*[a[n] for n, _ in df.attention._Cache._fields_])


Q, OUT, TAB, LEN, WS = (A + (i << 26) for i in range(1, 6))


def decode(df, c=None, **kw):
    a = dict(out=OUT, ob=8 * 64, oh=64, lse=None, q=Q, qb=8 * 64, qh=64, table=TAB, ts=4, cols=4, lens=LEN, batch=2,
             heads=8, max_len=64, scale=0.125, window=0, ws=WS, wsb=1 << 40, status=None)
    a.update(kw)
    c = cache(df) if c is None else c
    return df.attention.lib.detfold_attn_decode(
        a["out"], a["ob"], a["oh"], a["lse"], a["q"], a["qb"], a["qh"], ctypes.addressof(c) if c else None, a["table"],
        a["ts"], a["cols"], a["lens"], a["batch"], a["heads"], a["max_len"], a["scale"], a["window"], a["ws"], a["wsb"],
        a["status"], None)


@no_gpu_only
def test_decode_refusals(df):
    S = df.STATUS
    assert decode(df, c=False) == S["DETFOLD_ERR_NULL"]
    for name in ("out", "q", "table", "lens"):
        assert decode(df, **{name: None}) == S["DETFOLD_ERR_NULL"], name
    assert decode(df, c=cache(df, k=None)) == S["DETFOLD_ERR_NULL"]
    for bad in (dict(dtype=3), dict(dtype=-1), dict(num_pages=0), dict(page_size=0), dict(kv_heads=0), dict(head_dim=0),
                dict(head_dim=264), dict(page_stride=-8), dict(page_stride=1 << 62), dict(num_pages=1 << 60),
                dict(page_size=1 << 21)):
        assert decode(df, c=cache(df, **bad)) == S["DETFOLD_ERR_ARG"], bad
    for bad in (dict(batch=-1), dict(heads=0), dict(heads=7), dict(heads=-2), dict(window=-1), dict(ts=-1),
                dict(ob=-1), dict(qh=1 << 60), dict(cols=-1), dict(batch=1 << 20, heads=1 << 20)):
        assert decode(df, **bad) == S["DETFOLD_ERR_ARG"], bad
    for bad in (dict(max_len=-1), dict(max_len=65), dict(max_len=(1 << 30) + 1), dict(cols=3), dict(cols=0)):
        assert decode(df, **bad) == S["DETFOLD_ERR_LEN"], bad
    for bad in (dict(k=A + 8), dict(v=A + (1 << 24) + 2), dict(page_stride=16 * 2 * 64 + 4), dict(token_stride=129),
                dict(head_stride=65), dict(head_dim=60)):
        assert decode(df, c=cache(df, **bad)) == S["DETFOLD_ERR_ALIGN"], bad
    for bad in (dict(out=OUT + 1), dict(q=Q + 1), dict(lse=A + (7 << 26) + 2), dict(table=TAB + 2), dict(lens=LEN + 1),
                dict(status=A + (8 << 26) + 1)):
        assert decode(df, **bad) == S["DETFOLD_ERR_ALIGN"], bad
    assert decode(df, batch=0) == S["DETFOLD_OK"]
    for bad in (dict(out=Q), dict(out=A + 64), dict(lse=OUT + 64), dict(lse=LEN + 4), dict(out=TAB)):
        assert decode(df, **bad) == S["DETFOLD_ERR_OVERLAP"], bad


@no_gpu_only
def test_decode_workspace(df):
    S, F = df.STATUS, df.attention.lib.detfold_attn_decode_workspace_bytes
    c = cache(df)
    p = ctypes.addressof(c)
    assert F(None, 1, 8, 64) == S["DETFOLD_ERR_NULL"]
    assert F(p, -1, 8, 64) == S["DETFOLD_ERR_ARG"] and F(p, 1, 3, 64) == S["DETFOLD_ERR_ARG"]
    assert F(p, 1, 8, -1) == S["DETFOLD_ERR_LEN"]
    assert F(p, 0, 8, 64) >= 0 and F(p, 64, 8, 1 << 20) >= F(p, 64, 8, 64) >= 0
    big = cache(df, num_pages=1 << 20)
    need = F(ctypes.addressof(big), 2, 8, 100000)
    if need > 0:
        big_call = dict(max_len=100000, cols=6250, ts=6250)
        far = A + (1 << 42)
        place = dict(out=far, q=far + (1 << 30), table=far + (2 << 30), lens=far + (3 << 30))
        assert decode(df, c=big, **big_call, **place, ws=None) == S["DETFOLD_ERR_WORKSPACE"]
        assert decode(df, c=big, **big_call, **place, ws=far + (4 << 30), wsb=need - 1) == S["DETFOLD_ERR_WORKSPACE"]
        assert decode(df, c=big, **big_call, **place, ws=far + (4 << 30) + 8) == S["DETFOLD_ERR_WORKSPACE"]
        assert decode(df, c=big, **big_call, **place, ws=far) == S["DETFOLD_ERR_OVERLAP"]


@no_gpu_only
def test_workspace_grows_with_every_size(df):
    # no GPU needed: every type, tile and grouping, lengths around the chunk's and large ones
    F = df.attention.lib.detfold_attn_decode_workspace_bytes
    for dtype in (0, 1, 2):
        for head_dim in (8, 64, 80, 128, 256):
            c = cache(df, dtype=dtype, head_dim=head_dim, kv_heads=2, num_pages=1 << 20)
            for group in (1, 4, 9):
                for batch in (1, 152, 153, 229, 304, 305, 1000):
                    got = [F(ctypes.addressof(c), batch, 2 * group, n)
                           for n in (0, 1, 127, 128, 129, 256, 257, 384, 385, 1000, 1 << 14, 1 << 24)]
                    assert got == sorted(got) and got[0] >= 0, (dtype, head_dim, group, batch)


def append(df, c=None, rope="default", **kw):
    a = dict(k=Q, kt=128, kh=64, v=Q + (1 << 20), vt=128, vh=64, slots=TAB, tokens=3, pos=LEN, qo=OUT, ot=512, oh=64,
             q=WS, qt=512, qh=64, heads=8, status=None)
    a.update(kw)
    c = cache(df) if c is None else c
    r = df.attention._Rope(A + (9 << 26), 100, 64, 0) if rope == "default" else rope
    return df.attention.lib.detfold_kv_append(
        ctypes.addressof(c) if c else None, a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"], a["slots"], a["tokens"],
        ctypes.addressof(r) if r else None, a["pos"], a["qo"], a["ot"], a["oh"], a["q"], a["qt"], a["qh"], a["heads"],
        a["status"], None)


@no_gpu_only
def test_append_refusals(df):
    S, R = df.STATUS, df.attention._Rope
    assert append(df, c=False) == S["DETFOLD_ERR_NULL"]
    for name in ("k", "v", "slots", "pos", "q", "qo"):
        assert append(df, **{name: None}) == S["DETFOLD_ERR_NULL"], name
    assert append(df, rope=R(None, 100, 64, 0)) == S["DETFOLD_ERR_NULL"]
    T = A + (9 << 26)
    for bad in (R(T, 0, 64, 0), R(T, 100, 63, 0), R(T, 100, 0, 0), R(T, 100, 66, 0), R(T, 100, 64, 2)):
        assert append(df, rope=bad) == S["DETFOLD_ERR_ARG"]
    for bad in (dict(heads=-1), dict(heads=0), dict(kt=-1), dict(vh=-1), dict(qt=1 << 60), dict(ot=-4)):
        assert append(df, **bad) == S["DETFOLD_ERR_ARG"], bad
    assert append(df, tokens=-1) == S["DETFOLD_ERR_LEN"]
    for bad in (dict(k=Q + 1), dict(v=Q + 3), dict(slots=TAB + 4), dict(pos=LEN + 4), dict(q=WS + 1), dict(qo=OUT + 1),
                dict(status=A + 2)):
        assert append(df, **bad) == S["DETFOLD_ERR_ALIGN"], bad
    assert append(df, rope=R(T + 2, 100, 64, 0)) == S["DETFOLD_ERR_ALIGN"]
    for bad in (dict(k=A + 64), dict(v=A + (1 << 24)), dict(qo=A), dict(q=A + 2), dict(qo=WS + 128), dict(qo=Q)):
        assert append(df, **bad) == S["DETFOLD_ERR_OVERLAP"], bad
    assert append(df, qo=WS, ot=1024) == S["DETFOLD_ERR_OVERLAP"]  # in place, but laid out otherwise
    assert append(df, tokens=0) == S["DETFOLD_OK"]


@no_gpu_only
def test_join_refusals(df):
    S, F = df.STATUS, df.attention.lib.detfold_attn_join
    tab = lambda *p: (ctypes.c_void_p * len(p))(*p)  # noqa: E731
    parts, lses = tab(A, A + 4096), tab(A + 8192, A + 12288)
    out, lse = A + (1 << 20), A + (2 << 20)
    assert F(None, lse, parts, lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_NULL"]
    assert F(out, lse, None, lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_NULL"]
    assert F(out, lse, parts, None, 2, 4, 64, 1, None) == S["DETFOLD_ERR_NULL"]
    assert F(out, lse, tab(A, 0), lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_NULL"]
    assert F(out, lse, parts, lses, 0, 4, 64, 1, None) == S["DETFOLD_ERR_WORLD"]
    assert F(out, lse, parts, lses, 257, 4, 64, 1, None) == S["DETFOLD_ERR_WORLD"]
    assert F(out, lse, parts, lses, 2, 4, 64, 3, None) == S["DETFOLD_ERR_ARG"]
    assert F(out, lse, parts, lses, 2, 4, 0, 1, None) == S["DETFOLD_ERR_ARG"]
    assert F(out, lse, parts, lses, 2, -1, 64, 1, None) == S["DETFOLD_ERR_LEN"]
    assert F(out, lse, parts, lses, 2, 1 << 60, 64, 1, None) == S["DETFOLD_ERR_LEN"]
    assert F(out + 1, lse, parts, lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_ALIGN"]
    assert F(out, lse + 2, parts, lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_ALIGN"]
    assert F(out, lse, tab(A, A + 4097), lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_ALIGN"]
    assert F(out, lse, parts, tab(A + 8192, A + 12290), 2, 4, 64, 1, None) == S["DETFOLD_ERR_ALIGN"]
    assert F(A + 64, lse, parts, lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_OVERLAP"]
    assert F(A + 8192, lse, parts, lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_OVERLAP"]
    assert F(out, A + 8, parts, lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_OVERLAP"]
    assert F(out, out + 4, parts, lses, 2, 4, 64, 1, None) == S["DETFOLD_ERR_OVERLAP"]
    assert F(out, lse, parts, lses, 2, 0, 64, 1, None) == S["DETFOLD_OK"]


@no_gpu_only
def test_launch_without_device_reports_a_cuda_error(df):
    assert decode(df) == df.STATUS["DETFOLD_ERR_CUDA"]
    assert df.attention.detfold_attn_last_cuda_error() != 0


def test_binding_refuses_what_it_can_see(df):
    torch = pytest.importorskip("torch")
    k = torch.zeros(2, 4, 1, 8)
    with pytest.raises(TypeError):
        df.PagedCache(k, k)  # CPU tensors
    with pytest.raises(TypeError):
        df.PagedCache(k.to(torch.int32), k)
    with pytest.raises(TypeError):
        df.Rope(torch.zeros(4, 8))
    with pytest.raises(TypeError):
        df.detfold_attn_join(torch.zeros(2, 8), [torch.zeros(2, 8)], [torch.zeros(2)])
    with pytest.raises(ValueError):
        df.detfold_attn_join(torch.zeros(2, 8), [torch.zeros(2, 8)], [])
