"""The restated layout of a one-token attention call against the library's bytes, on the CPU."""
import ctypes

import pytest

from attn_plan import plan
from test_attn_abi import cache, df  # noqa: F401


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_bytes_are_the_library_s(df, dtype):  # noqa: F811
    F = df.attention.lib.detfold_attn_decode_workspace_bytes
    for head_dim in (8, 64, 72, 128, 136, 256):
        for kv in (1, 2, 8):
            for group in (1, 3, 8, 9, 16, 40):
                c = cache(df, dtype=dtype, head_dim=head_dim, kv_heads=kv, num_pages=1 << 20)
                for batch in (1, 37, 152, 153, 304, 305, 456, 457, 608, 609, 2000):
                    for n in (0, 1, 64, 128, 129, 256, 257, 512, 513, 900, 5000, 1 << 20, 1 << 30):
                        want = plan(4 if dtype == 0 else 2, batch, kv, group, head_dim, n)[2]
                        got = F(ctypes.addressof(c), batch, kv * group, n)
                        assert got == want, (head_dim, kv, group, batch, n)


def test_every_way_is_taken_on_both_sides_of_its_bounds():
    way = lambda *a: plan(2, *a)[0]  # noqa: E731
    assert [way(b, 1, 2, 64, 900) for b in (228, 229, 608, 609)] == ["chunk", "shares by pair", "shares by pair", "shares by CTA"]
    assert [way(b, 1, 2, 64, 512) for b in (152, 153, 1824, 1825)] == ["chunk", "pair", "pair", "shares by CTA"]
    assert [way(1000, 1, 2, 64, n) for n in (128, 129, 512, 513)] == ["one chunk", "pair", "pair", "shares by CTA"]
