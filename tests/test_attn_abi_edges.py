"""The attention library's C boundary on the CPU, further: calls without elements."""
import ctypes

import pytest

from test_attn_abi import A, LEN, OUT, Q, TAB, WS, append, cache, decode, df, no_gpu_only  # noqa: F401


@no_gpu_only
def test_operands_without_elements_need_no_address(df):  # noqa: F811
    S = df.STATUS
    none = dict(out=None, q=None, table=None, lens=None)
    assert decode(df, batch=0, **none) == S["DETFOLD_OK"]
    assert decode(df, batch=0, **none, cols=0, max_len=0, ws=None, wsb=0) == S["DETFOLD_OK"]
    assert append(df, tokens=0, k=None, v=None, slots=None, pos=None, q=None, qo=None) == S["DETFOLD_OK"]
    assert append(df, tokens=0, rope=False, k=None, v=None, slots=None, pos=None, q=None, qo=None, heads=0) == S["DETFOLD_OK"]
    tab = lambda *p: (ctypes.c_void_p * len(p))(*p)  # noqa: E731
    assert df.attention.lib.detfold_attn_join(None, None, tab(0, 0), tab(0, 0), 2, 0, 64, 1, None) == S["DETFOLD_OK"]


@no_gpu_only
@pytest.mark.parametrize("name", ["out", "q", "lens"])
def test_a_table_without_columns_excuses_the_table_only(df, name):  # noqa: F811
    S = df.STATUS
    assert decode(df, table=None, cols=0, max_len=0, **{name: None}) == S["DETFOLD_ERR_NULL"]
    assert decode(df, table=None, cols=1, max_len=0) == S["DETFOLD_ERR_NULL"]
    assert decode(df, table=None, cols=0, max_len=1) == S["DETFOLD_ERR_LEN"]


@no_gpu_only
def test_what_is_wrong_without_elements_is_refused(df):  # noqa: F811
    S = df.STATUS
    assert decode(df, batch=0, c=cache(df, k=None)) == S["DETFOLD_ERR_NULL"]
    assert decode(df, batch=0, heads=7) == S["DETFOLD_ERR_ARG"]
    assert append(df, tokens=0, c=cache(df, v=None)) == S["DETFOLD_ERR_NULL"]
    assert append(df, tokens=0, rope=df.attention._Rope(None, 100, 64, 0)) == S["DETFOLD_ERR_NULL"]
    assert append(df, tokens=-1, k=None) == S["DETFOLD_ERR_NULL"]
    tab = lambda *p: (ctypes.c_void_p * len(p))(*p)  # noqa: E731
    F = df.attention.lib.detfold_attn_join
    assert F(None, None, None, tab(0, 0), 2, 0, 64, 1, None) == S["DETFOLD_ERR_NULL"]
    assert F(None, None, tab(0, 0), tab(0, 0), 2, 4, 64, 1, None) == S["DETFOLD_ERR_NULL"]
    assert F(OUT, None, tab(A, 0), tab(LEN, WS), 2, 4, 64, 1, None) == S["DETFOLD_ERR_NULL"]
    assert F(OUT, None, tab(A, Q), tab(0, TAB), 2, 4, 64, 1, None) == S["DETFOLD_ERR_NULL"]


@no_gpu_only
def test_written_operands_whose_elements_share_addresses_are_refused(df):  # noqa: F811
    # two neighbours less than a head apart: their elements would be written twice, in any order
    S = df.STATUS
    for bad in (dict(ob=0), dict(ob=56), dict(oh=0), dict(oh=32), dict(oh=63)):
        assert decode(df, **bad) == S["DETFOLD_ERR_ARG"], bad
    for bad in (dict(page_stride=0), dict(token_stride=0), dict(head_stride=0), dict(page_stride=56), dict(token_stride=8),
                dict(head_stride=48)):
        assert append(df, c=cache(df, **bad)) == S["DETFOLD_ERR_ARG"], bad
    for bad in (dict(ot=0), dict(oh=0), dict(ot=63), dict(oh=1)):
        assert append(df, **bad) == S["DETFOLD_ERR_ARG"], bad
    assert append(df, qo=WS, ot=0, qt=0) == S["DETFOLD_ERR_ARG"]  # in place
    # one of a kind has no neighbour, whatever its stride; what is only read may be broadcast
    OK = (S["DETFOLD_OK"], S["DETFOLD_ERR_CUDA"])  # past the checks: no device to launch on
    assert decode(df, batch=1, ob=0) in OK and decode(df, qb=0, qh=0) in OK
    assert decode(df, c=cache(df, kv_heads=1, head_stride=0), heads=1, oh=0) in OK
    assert decode(df, c=cache(df, page_stride=0)) in OK
    assert append(df, c=cache(df, num_pages=1, page_stride=0)) in OK
    assert append(df, kt=0, kh=0, vt=0, qt=0) in OK and append(df, tokens=1, ot=0) in OK
