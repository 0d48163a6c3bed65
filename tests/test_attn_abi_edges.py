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
