"""One-token attention on both sides of every bound at which the work is shared out another
way: the way that the rules give is the one that the workspace shows, nothing behind the
workspace is written, and a sequence has the bits that it has alone.

The workspace is filled before the call: a CTA a pair writes none of it, a CTA a chunk no header
(the first 16 bytes a slot), shares write every header."""
import pytest
import torch

import attn_ref as ref
import deterministic_fixed_order_gb300 as df
from attn_plan import plan
from test_gpu_attn import BF16, F16, F32, Decode

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

ONE, PAIR, CHUNK, BY_PAIR, BY_CTA = "one chunk", "pair", "chunk", "shares by pair", "shares by CTA"


def rows(dtype, kv, group, head_dim, longest, window, *batches):
    return [(dtype, batch, kv, group, head_dim, longest, window, way) for batch, way in batches]


CASES = [
    # four CTAs an SM: 608 resident
    *rows(BF16, 1, 2, 64, 900, 0, (228, CHUNK), (229, BY_PAIR), (608, BY_PAIR), (609, BY_CTA)),
    *rows(F16, 3, 2, 64, 900, 0, (202, BY_PAIR), (203, BY_CTA)),
    *rows(BF16, 1, 2, 64, 900, 600, (364, CHUNK), (365, BY_PAIR), (608, BY_PAIR), (609, BY_CTA)),
    *rows(BF16, 1, 2, 8, 900, 500, (152, CHUNK), (153, PAIR), (609, PAIR), (1824, PAIR), (1825, BY_CTA)),
    *rows(BF16, 1, 2, 8, 900, 128, (609, ONE), (2000, ONE)),
    *rows(F16, 1, 2, 64, 512, 0, (1824, PAIR), (1825, BY_CTA)),
    # three: 456
    *rows(BF16, 1, 16, 64, 900, 0, (171, CHUNK), (172, BY_PAIR), (456, BY_PAIR), (457, BY_CTA)),
    *rows(F16, 3, 12, 64, 900, 0, (152, BY_PAIR), (153, BY_CTA)),
    *rows(BF16, 1, 9, 8, 900, 600, (273, CHUNK), (274, BY_PAIR), (457, BY_CTA)),
    *rows(BF16, 1, 16, 64, 512, 0, (1368, PAIR), (1369, BY_CTA)),
    # two: 304
    *rows(BF16, 1, 2, 128, 900, 0, (114, CHUNK), (115, BY_PAIR), (304, BY_PAIR), (305, BY_CTA)),
    *rows(F16, 1, 24, 128, 900, 0, (57, CHUNK), (58, BY_PAIR), (152, BY_PAIR), (153, BY_CTA)),
    *rows(BF16, 1, 2, 128, 900, 600, (182, CHUNK), (183, BY_PAIR), (304, BY_PAIR), (305, BY_CTA)),
    *rows(BF16, 1, 1, 72, 900, 512, (912, PAIR), (913, BY_CTA)),
    *rows(F16, 1, 2, 256, 900, 0, (114, CHUNK), (115, BY_PAIR), (304, BY_PAIR), (305, BY_CTA)),
    *rows(BF16, 1, 16, 136, 900, 300, (152, CHUNK), (153, BY_CTA)),
    *rows(BF16, 1, 1, 256, 256, 0, (912, PAIR), (913, BY_CTA)),
    *rows(F32, 1, 2, 128, 900, 0, (114, CHUNK), (115, BY_PAIR), (304, BY_PAIR), (305, BY_CTA)),
    *rows(F32, 1, 1, 64, 900, 600, (182, CHUNK), (183, BY_PAIR), (305, BY_CTA)),
    *rows(F32, 1, 6, 8, 512, 0, (912, PAIR), (913, BY_CTA)),
    *rows(F32, 1, 9, 256, 900, 0, (57, CHUNK), (58, BY_PAIR), (152, BY_PAIR), (153, BY_CTA)),
]


@pytest.mark.parametrize("dtype,batch,kv,group,head_dim,longest,window,way", CASES)
def test_a_sequence_has_its_own_bits_whichever_way_the_work_is_shared(dtype, batch, kv, group, head_dim, longest, window,
                                                                      way):
    bytes_each = 4 if dtype == F32 else 2
    got, slots, used = plan(bytes_each, batch, kv, group, head_dim, min(window or longest, longest))
    assert got == way
    lens = [0 if b % 11 == 5 else longest // 3 + (53 * b) % (longest - longest // 3 + 1) for b in range(batch)]
    lens[batch // 2] = longest
    d = Decode(dtype, lens, kv * group, kv, head_dim, 16, window=window, cols=-(-longest // 16))
    need = df.detfold_attn_decode_workspace_bytes(d.cache, batch, kv * group, longest)
    assert need == plan(bytes_each, batch, kv, group, head_dim, longest)[2] >= used
    some = [0, 5, batch // 2, batch - 1]
    want, wlse, tol, ltol = ref.decode(d.q[some], d.k, d.v, d.table[some], [lens[b] for b in some], d.scale, window)
    for fill in (0, 255):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(d.q), torch.empty(d.q.shape[:2], device="cuda")
        df.detfold_attn_decode(out, d.q, d.cache, d.table, d.lens, longest, d.scale, window=window, lse=lse,
                               workspace=ws[:need])
        torch.cuda.synchronize()
        ref.assert_near(out[some], want, tol, way)
        ref.assert_near(lse[some], wlse, ltol, way + " lse")
        assert bool((ws[used:] == fill).all()), "nothing behind what the layout needs"
        if fill == 255:
            headers = (ws[:16 * slots].view(slots, 16) != fill).any(1) if slots else torch.zeros(0)
            wrote = bool((ws[:used] != fill).any())
            shown = {ONE: not wrote, PAIR: not wrote, CHUNK: wrote and not bool(headers.any()),
                     BY_PAIR: bool(headers.all()), BY_CTA: bool(headers.all())}
            assert shown[way], f"the workspace does not show {way}"
        for b in some[1:]:
            alone, alone_lse = torch.empty_like(d.q[:1]), torch.empty_like(lse[:1])
            df.detfold_attn_decode(alone, d.q[b:b + 1], d.cache, d.table[b:b + 1], d.lens[b:b + 1], longest, d.scale,
                                   window=window, lse=alone_lse, workspace=ws[:need])
            assert torch.equal(alone[0], out[b]) and torch.equal(alone_lse[0], lse[b]), b


@pytest.mark.parametrize("batch", [261, 608, 609, 1825])
def test_the_bytes_of_max_len_hold_for_every_window(batch):
    # one workspace, asked for once: windows below max_len lay it out otherwise, and stay inside
    lens = [300 + (7 * b) % 601 for b in range(batch)]
    d = Decode(BF16, lens, 2, 1, 8, 16)
    need = df.detfold_attn_decode_workspace_bytes(d.cache, batch, 2, d.max_len)
    seen = set()
    for window in (0, 100, 129, 257, 400, 512, 513, 600, 650, 800, 899):
        way, slots, used = plan(2, batch, 1, 2, 8, min(window or d.max_len, d.max_len))
        seen.add(way)
        assert used <= need
        ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(d.q)
        df.detfold_attn_decode(out, d.q, d.cache, d.table, d.lens, d.max_len, d.scale, window=window, workspace=ws[:need])
        torch.cuda.synchronize()
        assert bool((ws[used:] == 255).all()), window
        assert bool((ws[:used] != 255).any()) == (way not in (ONE, PAIR)), (window, way)
        some = [0, batch // 2, batch - 1]
        want, _, tol, _ = ref.decode(d.q[some], d.k, d.v, d.table[some], [lens[b] for b in some], d.scale, window)
        ref.assert_near(out[some], want, tol, f"window {window}")
    assert seen == {261: {ONE, PAIR, CHUNK, BY_PAIR}, 608: {ONE, PAIR, BY_PAIR},
                    609: {ONE, PAIR, BY_CTA}, 1825: {ONE, BY_CTA}}[batch]
