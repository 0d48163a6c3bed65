"""The decode-step operators on the GPU against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import attn_ref as ref

import deterministic_fixed_order_gb300 as df

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
ERR_ARG = df.STATUS["DETFOLD_ERR_ARG"]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


class Decode:
    """A pool with the sequences' pages anywhere in it; every row that no token
    was written to holds NaN, every table entry that is not needed -1."""

    def __init__(self, dtype, lens, hq, hk, width, page, window=0, layout="token", seed=1, cols=None,
                 q_scale=1.5, spare=2):
        g = gen(seed)
        self.lens_host, self.window, self.scale = list(lens), window, width ** -0.5
        batch, self.max_len = len(lens), max(list(lens) + [1])
        cols = cols or -(-self.max_len // page)
        col = torch.arange(cols, device="cuda")
        n = torch.tensor(lens, device="cuda")
        first = (n - window).clamp(min=0) if window else torch.zeros_like(n)
        held = (col * page < n[:, None]) & ((col + 1) * page > first[:, None])
        count = int(held.sum())
        pages = count + spare
        self.table = torch.full((batch, cols), -1, dtype=torch.int32, device="cuda")
        order = torch.randperm(pages, generator=g, device="cuda")[:count]
        self.table[held] = order.to(torch.int32)
        if layout == "token":
            k, v = (randn(g, (pages, page, hk, width), dtype) for _ in range(2))
        elif layout == "head":
            k, v = (randn(g, (pages, hk, page, width), dtype).transpose(1, 2) for _ in range(2))
        else:  # one buffer holds both
            both = randn(g, (pages, 2, page, hk, width), dtype)
            k, v = both[:, 0], both[:, 1]
        written = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
        rows = col[:, None] * page + torch.arange(page, device="cuda")
        written[order] = (rows < n[:, None, None])[held]
        k[~written], v[~written] = float("nan"), float("nan")
        self.q = randn(g, (batch, hq, width), dtype, q_scale)
        self.k, self.v, self.lens = k, v, n.to(torch.int32)
        self.cache = df.PagedCache(k, v)

    def run(self, q=None, table=None, lens=None, status=None, max_len=None, stream=None, out=None, window=None):
        q = self.q if q is None else q
        lens = self.lens if lens is None else lens
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda") if out is None else out
        lse = torch.empty(q.shape[:2], dtype=F32, device="cuda")
        max_len = self.max_len if max_len is None else max_len
        need = df.detfold_attn_decode_workspace_bytes(self.cache, q.shape[0], q.shape[1], max_len)
        ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")  # NaN as any float
        df.detfold_attn_decode(out, q, self.cache, self.table if table is None else table, lens, max_len,
                               self.scale, window=self.window if window is None else window, lse=lse,
                               workspace=ws, status=status, stream=stream)
        torch.cuda.synchronize()
        assert bool((ws[need:] == 255).all())
        return out, lse

    def check(self, what, rows=None):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = self.run(status=status)
        assert int(status) == 0
        want, wlse, tol, ltol = ref.decode(self.q, self.k, self.v, self.table, self.lens_host, self.scale, self.window)
        ref.assert_near(out, want, tol, what + " out")
        ref.assert_near(lse, wlse, ltol, what + " lse")
        return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257, 511]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("hq,hk,width", [(1, 1, 64), (8, 8, 64), (8, 1, 128), (12, 4, 80), (7, 1, 96), (16, 1, 128),
                                         (10, 2, 32), (4, 2, 256), (40, 2, 64), (9, 1, 192), (24, 1, 256),
                                         (3, 3, 8), (4, 1, 200)])
def test_decode_matches_the_definition(dtype, hq, hk, width):
    Decode(dtype, EDGES, hq, hk, width, 16).check(f"{dtype} {hq}/{hk}x{width}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 256])
@pytest.mark.parametrize("layout", ["token", "head", "both"])
def test_decode_page_sizes_and_layouts(dtype, page, layout):
    Decode(dtype, [1, 5, 70, 333, 0, 200], 8, 2, 64, page, layout=layout).check(f"page {page} {layout}")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("window", [1, 7, 64, 100, 1000])
def test_decode_window(dtype, window):
    Decode(dtype, [0, 1, 7, 8, 99, 100, 101, 500, 1500], 8, 4, 128, 24, window=window).check(f"window {window}")


@pytest.mark.parametrize("dtype,hq,hk,width", [(BF16, 32, 8, 128), (F16, 8, 1, 128), (F32, 4, 4, 64), (BF16, 16, 4, 256)])
@pytest.mark.parametrize("lens", [[4093], [1, 9000, 0, 17, 2049], [12345, 12345]])
def test_decode_long_and_split(dtype, hq, hk, width, lens):
    Decode(dtype, lens, hq, hk, width, 16).check(f"{lens}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_many_sequences(dtype):
    r = np.random.RandomState(7)
    lens = [int(x) for x in np.exp(r.uniform(0, np.log(700), 200))] + [0, 900]
    Decode(dtype, lens, 4, 2, 64, 8).check("many")


def test_decode_no_tokens_at_all():
    d = Decode(BF16, [0, 0, 0], 8, 2, 128, 16)
    out, lse = d.run()
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    out, lse = d.run(max_len=0, window=0)
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())


@pytest.mark.parametrize("dtype,hq,hk,width,window", [(BF16, 32, 8, 128, 0), (F32, 8, 8, 64, 0), (F16, 16, 1, 256, 0),
                                                      (BF16, 8, 1, 128, 777)])
def test_decode_bits_do_not_depend_on_the_batch_or_the_pages(dtype, hq, hk, width, window):
    lens = [5000, 3, 130, 2000, 1, 0, 700, 1025]
    d = Decode(dtype, lens, hq, hk, width, 16, window=window)
    out, lse = d.run()
    again, lse2 = d.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    for b in range(len(lens)):  # alone
        o, s = d.run(q=d.q[b:b + 1], table=d.table[b:b + 1], lens=d.lens[b:b + 1])
        assert torch.equal(o[0], out[b]) and torch.equal(s[0], lse[b]), b
    # with a larger bound on the lengths, other neighbours and another order
    pick = torch.tensor([3, 0, 0, 7, 2] * 9, device="cuda")
    table = torch.full((len(pick), d.table.shape[1] + 300), -1, dtype=torch.int32, device="cuda")
    table[:, :d.table.shape[1]] = d.table[pick]
    o, s = d.run(q=d.q[pick].contiguous(), table=table, lens=d.lens[pick].contiguous(), max_len=table.shape[1] * 16)
    assert torch.equal(o, out[pick]) and torch.equal(s, lse[pick])
    # the same tokens in other pages
    pages = d.k.shape[0]
    move = torch.randperm(pages, generator=gen(5), device="cuda")
    k, v = torch.empty_like(d.k), torch.empty_like(d.v)
    k[move], v[move] = d.k, d.v
    d.cache = df.PagedCache(k, v)
    moved = torch.where(d.table >= 0, move[d.table.clamp(min=0).long()].to(torch.int32), d.table)
    o, s = d.run(table=moved)
    assert torch.equal(o, out) and torch.equal(s, lse)


def test_decode_strided_views_touch_nothing_else():
    d = Decode(BF16, [300, 17], 8, 2, 64, 16)
    want, _ = d.run()
    wide = torch.full((2, 12, 72), 7.0, dtype=BF16, device="cuda")
    out = wide[:, 3:11, 5:69]  # rows at odd offsets
    fused = torch.zeros((2, 20, 65), dtype=BF16, device="cuda")
    q = fused[:, 1:9, 1:]
    q.copy_(d.q)
    df_out, _ = d.run(q=q, out=out)
    assert torch.equal(out, want)
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[:, 3:11, 5:69] = False
    assert bool((wide[keep] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_extreme_scores(dtype):
    # weights of one token only; all scores far below zero; scores that differ by more than exp can hold
    d = Decode(dtype, [200, 200, 200], 2, 1, 64, 16)
    d.q[1] = 0
    d.q[1, :, 0] = -1e15
    d.k[d.table[1][:13].long(), :, :, 0] = 1e15  # every score is -1e30 / 8
    d.q[2] *= 60
    d.v[torch.isnan(d.v)] = 0
    d.k[torch.isnan(d.k)] = 0
    out, lse = d.run()
    want, wlse, tol, ltol = ref.decode(d.q, d.k, d.v, d.table, [200] * 3, d.scale)
    for b in (0, 2):
        ref.assert_near(out[b], want[b], tol[b], f"row {b}")
        ref.assert_near(lse[b], wlse[b], ltol[b], f"row {b} lse")
    assert bool(torch.isfinite(out[1]).all()) and bool((lse[1] < -1e28).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_infinite_scores_and_values_follow_the_definition(dtype):
    # one key gives a score of -inf: it has no weight
    d = Decode(dtype, [100, 40], 2, 1, 64, 16)
    d.q[:, :, 0] = 1
    page = d.table[0, 2].long()
    d.k[page, 5, 0, 0] = float("-inf")
    out, lse = d.run()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    keep = torch.ones(100, dtype=torch.bool)
    keep[2 * 16 + 5] = False
    t = torch.arange(100)[keep].cuda()
    kk = d.k[d.table[0][t // 16].long(), t % 16][:, 0].double().cpu()
    s = (kk @ d.q[0, 0].double().cpu()) * d.scale
    assert abs(float(lse[0, 0]) - float(torch.logsumexp(s, 0))) < 1e-4


def test_decode_offsets_past_32_bits():
    # a pool of 2^31 + elements each for keys and values; the pages in use lie at its end
    width, page, hk = 128, 64, 8
    per_page = page * hk * width
    pages = (1 << 31) // per_page + 9
    k = torch.empty((pages, page, hk, width), dtype=BF16, device="cuda")
    v = torch.empty((pages, page, hk, width), dtype=BF16, device="cuda")
    g = gen(3)
    last = torch.arange(pages - 8, pages, device="cuda")
    k[last], v[last] = randn(g, (8, page, hk, width), BF16), randn(g, (8, page, hk, width), BF16)
    d = Decode(BF16, [500], 32, hk, width, page)
    d.k, d.v, d.cache = k, v, df.PagedCache(k, v)
    d.table = last[torch.randperm(8, generator=g, device="cuda")].to(torch.int32)[None]
    d.check("past 2^31 elements")


def test_decode_bad_indices_are_reported_and_kept_apart():
    d = Decode(BF16, [100, 300, 64, 300, 50], 8, 2, 64, 16)
    good, glse = d.run()
    for what, row, change in (("page below", 1, -1), ("page above", 1, d.k.shape[0]), ("far page", 3, 1 << 30)):
        table = d.table.clone()
        table[row, 4] = change
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = d.run(table=table, status=status)
        assert int(status) == ERR_ARG, what
        rest = [b for b in range(5) if b != row]
        assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], glse[rest]), what
        assert bool(torch.isnan(out[row]).all()) and bool(torch.isnan(lse[row]).all()), what
    for n in (-1, 301, -(1 << 31), (1 << 31) - 1):
        lens = d.lens.clone()
        lens[2] = n
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = d.run(lens=lens, status=status)
        assert int(status) == ERR_ARG, n
        rest = [0, 1, 3, 4]
        assert torch.equal(out[rest], good[rest]) and bool(torch.isnan(out[2]).all()), n
        d.run(lens=lens)  # without a status word
    # the word keeps an earlier report
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    d.run(status=status)
    assert int(status) == 5


def test_decode_on_another_stream_and_in_a_graph():
    d = Decode(BF16, [3000, 40, 500], 32, 8, 128, 16)
    want, wlse = d.run()
    side = torch.cuda.Stream()
    out, lse = d.run(stream=side)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    need = df.detfold_attn_decode_workspace_bytes(d.cache, 3, 32, d.max_len)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    lens, out, lse = d.lens.clone(), torch.empty_like(d.q), torch.empty((3, 32), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        df.detfold_attn_decode(out, d.q, d.cache, d.table, lens, d.max_len, d.scale, lse=lse, workspace=ws)
    for lengths in ([3000, 40, 500], [17, 0, 499], [2999, 1, 64]):
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        o, s = d.run(lens=lens)
        assert torch.equal(o, out) and torch.equal(s, lse), lengths


def test_decode_calls_in_a_row_share_a_workspace():
    a, b = Decode(BF16, [3000, 40], 32, 8, 128, 16, seed=1), Decode(BF16, [2500, 90], 32, 8, 128, 16, seed=2)
    want = [a.run()[0], b.run()[0]]
    need = df.detfold_attn_decode_workspace_bytes(a.cache, 2, 32, 3000)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(a.q) for _ in range(12)]
    for i, o in enumerate(outs):
        d = (a, b)[i % 2]
        df.detfold_attn_decode(o, d.q, d.cache, d.table, d.lens, d.max_len, d.scale, workspace=ws)
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2]), i


# ------------------------------------------------------------------ append

class Append:
    def __init__(self, dtype, tokens, hq, hk, width, rot, interleaved, page=16, layout="token", seed=1, fused=True,
                 positions=400):
        g = gen(seed)
        pages = -(-tokens // page) + 3
        if layout == "token":
            self.k, self.v = (randn(g, (pages, page, hk, width), dtype) for _ in range(2))
        else:
            self.k, self.v = (randn(g, (pages, hk, page, width), dtype).transpose(1, 2) for _ in range(2))
        qkv = randn(g, (tokens, hq + 2 * hk, width), dtype)
        self.q, self.nk, self.nv = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        self.cos_sin = torch.randn((positions, max(2, rot)), generator=g, device="cuda")
        self.rot, self.interleaved = rot, interleaved
        self.positions = torch.randint(0, positions, (tokens,), generator=g, device="cuda")
        self.slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
        self.cache = df.PagedCache(self.k, self.v)
        self.rope = df.Rope(self.cos_sin, interleaved) if rot else None

    def check(self, what, q_out=None, status_want=0):
        k0, v0 = self.k.clone(), self.v.clone()
        q0 = self.q.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.empty(self.q.shape, dtype=self.q.dtype, device="cuda") if q_out is None else q_out
        df.detfold_kv_append(self.cache, self.nk, self.nv, self.slots, rope=self.rope, positions=self.positions,
                             q=self.q if self.q.shape[1] else None, q_out=q_out if self.q.shape[1] else None,
                             status=status)
        torch.cuda.synchronize()
        assert int(status) == status_want, what
        page, total = self.k.shape[1], self.k.shape[0] * self.k.shape[1]
        live = (self.slots >= 0) & (self.slots < total)
        at = (self.slots[live] // page, self.slots[live] % page)
        if self.rot:
            ok = (self.positions >= 0) & (self.positions < self.cos_sin.shape[0])
            pos = torch.where(ok, self.positions, 0)
            wq, tq = ref.rotate(q0, self.cos_sin, pos, self.rot, self.interleaved)
            wk, tk = ref.rotate(self.nk, self.cos_sin, pos, self.rot, self.interleaved)
            for w in (wq, wk):
                w[..., :self.rot][~ok.cpu()] = float("nan")
            ref.assert_near(q_out, wq, tq, what + " q")
            ref.assert_near(self.k[at], wk[live.cpu()], tk[live.cpu()], what + " k")
            assert torch.equal(q_out[..., self.rot:], q0[..., self.rot:])
            assert torch.equal(self.k[at][..., self.rot:], self.nk[live][..., self.rot:])
        else:
            assert torch.equal(q_out, q0) and torch.equal(self.k[at], self.nk[live])
        assert torch.equal(self.v[at], self.nv[live])
        k0[at], v0[at] = self.k[at], self.v[at]
        same = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())  # noqa: E731
        assert same(self.k, k0) and same(self.v, v0), what + ": other rows changed"
        return q_out


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("width,rot", [(64, 64), (128, 128), (128, 64), (256, 64), (80, 80), (96, 24), (80, 20), (128, 2),
                                       (7, 4), (33, 32), (128, 0)])
def test_append_matches_the_definition(dtype, interleaved, width, rot):
    for tokens in (1, 5, 130):
        Append(dtype, tokens, 4, 2, width, rot, interleaved).check(f"{dtype} {width}/{rot} {tokens}")


@pytest.mark.parametrize("hq,hk", [(32, 8), (1, 1), (8, 1), (0, 4), (71, 1), (3, 3)])
@pytest.mark.parametrize("page,layout", [(16, "head"), (1, "token"), (24, "token"), (64, "head")])
def test_append_heads_and_pages(hq, hk, page, layout):
    Append(BF16, 77, hq, hk, 64, 64, False, page, layout).check(f"{hq}/{hk} page {page} {layout}")
    Append(BF16, 1, hq, hk, 64, 64, True, page, layout).check(f"{hq}/{hk} page {page} {layout} one")


def test_append_prompt():
    Append(BF16, 3001, 32, 8, 128, 128, False).check("prompt")
    Append(F32, 1023, 8, 8, 64, 32, True, layout="head").check("prompt f32")


def test_append_in_place_queries():
    for width, rot, il in ((128, 128, False), (128, 128, True), (80, 20, False)):
        want = Append(BF16, 50, 8, 2, width, rot, il).check("apart")
        a = Append(BF16, 50, 8, 2, width, rot, il)
        k0, v0 = a.nk.clone(), a.nv.clone()
        a.check("in place", q_out=a.q)
        assert torch.equal(a.q, want) and torch.equal(a.nk, k0) and torch.equal(a.nv, v0)


@pytest.mark.parametrize("width", [128, 80])
def test_append_misaligned_operands(width):
    a = Append(BF16, 20, 8, 2, width, width, False)
    buf = torch.zeros((20, 12, width + 3), dtype=BF16, device="cuda")
    view = buf[:, :, 1:width + 1]
    view[:, :8], view[:, 8:10], view[:, 10:] = a.q, a.nk, a.nv
    a.q, a.nk, a.nv = view[:, :8], view[:, 8:10], view[:, 10:]
    a.check("odd offsets")
    # a cache at an odd offset
    flat = torch.zeros(2 * 10 * 16 * 2 * width + 9, dtype=BF16, device="cuda")
    n = 10 * 16 * 2 * width
    b = Append(BF16, 20, 8, 2, width, width, True)
    b.k, b.v = flat[3:3 + n].view(10, 16, 2, width), flat[5 + n:5 + 2 * n].view(10, 16, 2, width)
    b.slots = b.slots % 160
    b.slots = torch.randperm(160, device="cuda")[:20]
    b.cache = df.PagedCache(b.k, b.v)
    b.check("odd cache")
    assert bool((flat[:3] == 0).all()) and bool((flat[3 + n:5 + n] == 0).all()) and bool((flat[5 + 2 * n:] == 0).all())


def test_append_padding_and_bad_indices():
    a = Append(BF16, 40, 4, 2, 64, 64, False)
    a.slots[30:] = -1
    a.slots[5] = -(1 << 62)
    a.check("padding")
    for slot in (a.k.shape[0] * 16, 1 << 40, (1 << 63) - 1):
        a = Append(BF16, 40, 4, 2, 64, 64, False)
        a.slots[7] = slot
        a.check("slot past the cache", status_want=ERR_ARG)
    for pos in (-1, 400, 1 << 40, -(1 << 63)):
        a = Append(BF16, 40, 4, 2, 64, 32, True)
        a.positions[9] = pos
        a.check("position outside the table", status_want=ERR_ARG)


def test_append_copies_every_value_unchanged():
    # values pass through as they are: NaN, infinities, signed zeros, subnormals
    a = Append(BF16, 16, 2, 2, 64, 0, False)
    special = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 1e-40, 0.0], dtype=BF16, device="cuda")
    a.nv[:, :, :6] = special
    a.nk[:, :, -6:] = special
    df.detfold_kv_append(a.cache, a.nk, a.nv, a.slots)
    torch.cuda.synchronize()
    at = (a.slots // 16, a.slots % 16)
    assert torch.equal(a.v[at].view(torch.int16), a.nv.contiguous().view(torch.int16))
    assert torch.equal(a.k[at].view(torch.int16), a.nk.contiguous().view(torch.int16))


def test_append_offsets_past_32_bits():
    width, hk, page = 128, 8, 16
    pages = (1 << 31) // (page * hk * width) + 4
    k = torch.empty((pages, page, hk, width), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    k[-3:], v[-3:] = 0, 0
    a = Append(BF16, 3, 8, hk, width, width, False)
    df.detfold_kv_append(a.cache, a.nk, a.nv, a.slots, rope=a.rope, positions=a.positions)
    at = (a.slots // page, a.slots % page)
    slots = pages * page - 1 - torch.arange(3, device="cuda") * 17
    df.detfold_kv_append(df.PagedCache(k, v), a.nk, a.nv, slots, rope=a.rope, positions=a.positions)
    torch.cuda.synchronize()
    far = (slots // page, slots % page)
    assert torch.equal(k[far], a.k[at]) and torch.equal(v[far], a.v[at])


# ------------------------------------------------------------------ join

def join_inputs(dtype, world, shape, width, seed=1, empty=0.15):
    g = gen(seed)
    parts = [randn(g, shape + (width,), dtype) for _ in range(world)]
    lses = [torch.randn(shape, generator=g, device="cuda") * 3 + 5 for _ in range(world)]
    for r in range(world):
        gone = torch.rand(shape, generator=g, device="cuda") < empty
        lses[r][gone] = float("-inf")
        parts[r][gone] = float("nan")
    return parts, lses


def check_join(parts, lses, what, out=None):
    shape = parts[0].shape
    want, wlse, tol, ltol = ref.join(parts, lses)
    out = torch.empty(shape, dtype=parts[0].dtype, device="cuda") if out is None else out
    lse = torch.empty(shape[:-1], dtype=F32, device="cuda")
    df.detfold_attn_join(out, parts, lses, lse=lse)
    torch.cuda.synchronize()
    ref.assert_near(out, want, tol, what)
    ref.assert_near(lse, wlse, ltol, what + " lse")
    return out, lse


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("world", [1, 2, 3, 4, 5, 8, 9, 17, 256])
@pytest.mark.parametrize("width", [128, 64, 80, 7, 1, 256, 1000])
def test_join_matches_the_definition(dtype, world, width):
    for shape in ((1,), (13, 5), (129, 3)):
        check_join(*join_inputs(dtype, world, shape, width), f"{dtype} W={world} {shape}x{width}")


def test_join_rows_that_are_empty_everywhere():
    parts, lses = join_inputs(BF16, 4, (50,), 128, empty=0.0)
    for r in range(4):
        lses[r][10:20] = float("-inf")
        parts[r][10:20] = float("nan")
    out, lse = check_join(parts, lses, "empty rows")
    assert bool((out[10:20] == 0).all()) and bool((lse[10:20] == float("-inf")).all())


def test_join_in_place_and_misaligned():
    parts, lses = join_inputs(F16, 3, (40, 8), 128)
    want, _ = check_join([p.clone() for p in parts], lses, "apart")
    for k in range(3):
        mine = [p.clone() for p in parts]
        df.detfold_attn_join(mine[k], mine, lses)
        torch.cuda.synchronize()
        assert torch.equal(mine[k], want), k
    shifted = []
    for r, p in enumerate(parts):
        buf = torch.zeros(p.numel() + 16, dtype=F16, device="cuda")
        view = buf[r + 1:r + 1 + p.numel()].view(p.shape)
        view.copy_(p)
        shifted.append(view)
    guard = torch.full((parts[0].numel() + 16,), 3.0, dtype=F16, device="cuda")
    out = guard[5:5 + parts[0].numel()].view(parts[0].shape)
    df.detfold_attn_join(out, shifted, lses)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert bool((guard[:5] == 3).all()) and bool((guard[5 + parts[0].numel():] == 3).all())


def test_join_extreme_weights():
    parts, lses = join_inputs(F32, 3, (6,), 32, empty=0.0)
    lses[0][:] = torch.tensor([1e30, -1e30, 3e38, -3e38, 0.0, 88.0], device="cuda")
    lses[1][:] = torch.tensor([1e30, -1e30, -3e38, -3e38, -200.0, -60.0], device="cuda")
    lses[2][:] = float("-inf")
    check_join(parts, lses, "extreme")


def test_join_offsets_past_32_bits():
    rows, width = (1 << 31) // 128 + 5, 128
    parts = [torch.full((rows, width), float(r + 1), dtype=BF16, device="cuda") for r in range(2)]
    lses = [torch.zeros(rows, device="cuda") for _ in range(2)]
    parts[0][-3:] = 5.0
    out, lse = torch.empty_like(parts[0]), torch.empty(rows, device="cuda")
    df.detfold_attn_join(out, parts, lses, lse=lse)
    torch.cuda.synchronize()
    assert bool((out[-3:] == 3.5).all()) and bool((out[:-3] == 1.5).all())
    assert bool(((lse - 0.6931472).abs() < 1e-6).all())


def test_split_attention_joins_to_the_whole():
    # each of three ranks attends to its own third of the tokens; the join gives the whole's attention
    d = Decode(F32, [90, 3, 60], 8, 2, 64, 10)
    want, wlse, tol, ltol = ref.decode(d.q, d.k, d.v, d.table, d.lens_host, d.scale)
    parts, lses = [], []
    for r in range(3):
        lens = (d.lens - 30 * r).clamp(0, 30)
        table = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
        table[:, :3] = d.table[:, 3 * r:3 * r + 3]
        o, s = d.run(table=table, lens=lens, max_len=30)
        parts.append(o)
        lses.append(s)
    out, lse = torch.empty_like(d.q), torch.empty((3, 8), device="cuda")
    df.detfold_attn_join(out, parts, lses, lse=lse)
    torch.cuda.synchronize()
    ref.assert_near(out, want, 4 * tol, "joined")
    ref.assert_near(lse, wlse, 4 * ltol, "joined lse")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_decode_one_token_outweighs_many(dtype):
    # One token's weight is e^14 times each other's, but 20000 others have a fiftieth of it together,
    # and the one's value is 0: the output is theirs, and no weight may lose its bits for being small.
    n, width = 20000, 64
    d = Decode(dtype, [n], 1, 1, width, 16, q_scale=0.0)
    d.q[0, 0, 0] = 8.0
    d.k[torch.isnan(d.k)] = 0
    d.k[..., 0] = 0
    page = d.table[0, 100].long()
    d.k[page, 3, 0, 0] = 14.0  # its score: 8 x 14 / sqrt(64)
    d.v.fill_(1.0)
    d.v[page, 3, 0] = 0
    out, lse = d.run()
    others = (n - 1) * torch.exp(torch.tensor(-14.0, dtype=torch.float64))
    want = (others / (1 + others)).expand(1, 1, width)
    # the weights' sum and the values' sum: n / 16 + 64 roundings of 2^-23, the weights' split 2^-16, the last rounding
    tol = want.abs() * (2 * (n / 16 + 64) * 2.0 ** -23 + 2.0 ** -15) + ref.final_round(want, dtype)
    ref.assert_near(out, want, tol, "sink")


def test_decode_bound_on_lengths_past_32_bits_of_work():
    # max_len 2^30: the shares' line is longer than 32 bits hold, the lengths themselves are short
    page, batch = 1 << 20, 40
    lens = [int(x) for x in np.random.RandomState(3).randint(0, 3000, batch)]
    g = gen(4)
    k, v = (randn(g, (batch, page, 1, 8), BF16) for _ in range(2))
    d = Decode(BF16, [1] * batch, 4, 1, 8, 16)
    d.k, d.v, d.cache, d.lens_host, d.max_len = k, v, df.PagedCache(k, v), lens, 1 << 30
    d.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    d.table = torch.full((batch, 1024), -1, dtype=torch.int32, device="cuda")
    d.table[:, 0] = torch.randperm(batch, generator=g, device="cuda").to(torch.int32)
    d.check("bound of 2^30 tokens")


@pytest.mark.parametrize("batch,heads", [(400, 1), (456, 1), (150, 3), (305, 1), (304, 1)])
def test_decode_workspace_suffices_whatever_the_window(batch, heads):
    # the bytes asked for max_len hold for every window: the guard behind them stays whole
    lens = [300 + (7 * b) % 85 for b in range(batch)]
    d = Decode(BF16, lens, 2 * heads, heads, 8, 16)
    need = df.detfold_attn_decode_workspace_bytes(d.cache, batch, 2 * heads, d.max_len)
    for window in (0, 129, 200, 256, 257, 300):
        ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(d.q)
        df.detfold_attn_decode(out, d.q, d.cache, d.table, d.lens, d.max_len, d.scale, window=window, workspace=ws[:need])
        torch.cuda.synchronize()
        assert bool((ws[need:] == 255).all()), window
        some = [0, batch // 2, batch - 1]
        want, _, tol, _ = ref.decode(d.q[some], d.k, d.v, d.table[some], [lens[b] for b in some], d.scale, window)
        ref.assert_near(out[some], want, tol, f"window {window}")


@pytest.mark.parametrize("batch,heads,group,head_dim", [
    (608, 1, 2, 64), (609, 1, 2, 64), (203, 3, 2, 64), (1900, 1, 2, 8),        # four CTAs an SM
    (456, 1, 16, 64), (457, 1, 16, 64), (1400, 1, 9, 8), (153, 3, 12, 64),     # three
    (304, 1, 12, 128), (305, 1, 2, 128), (153, 2, 8, 200), (920, 1, 1, 136)])  # two
def test_decode_at_the_counts_of_resident_ctas(batch, heads, group, head_dim):
    # slots by pairs and by CTAs, a CTA a chunk and shares, on both sides of each change; garbage in the workspace
    lens = [0 if b % 11 == 5 else 140 + (53 * b) % 250 for b in range(batch)]
    d = Decode(BF16, lens, group * heads, heads, head_dim, 16)
    need = df.detfold_attn_decode_workspace_bytes(d.cache, batch, group * heads, d.max_len)
    some = [0, 5, batch // 2, batch - 1]
    want, _, tol, _ = ref.decode(d.q[some], d.k, d.v, d.table[some], [lens[b] for b in some], d.scale)
    alone = torch.empty_like(d.q[:1])
    for fill in (0, 255):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(d.q)
        df.detfold_attn_decode(out, d.q, d.cache, d.table, d.lens, d.max_len, d.scale, workspace=ws[:need])
        torch.cuda.synchronize()
        assert bool((ws[need:] == fill).all())
        ref.assert_near(out[some], want, tol, f"workspace of {fill}")
        for b in (some[2], some[3]):
            df.detfold_attn_decode(alone, d.q[b:b + 1].contiguous(), d.cache, d.table[b:b + 1].contiguous(),
                                   d.lens[b:b + 1].contiguous(), d.max_len, d.scale, workspace=ws[:need])
            assert torch.equal(alone[0], out[b]), b


@pytest.mark.parametrize("longest", [129, 256, 300, 384, 512, 513, 700])
@pytest.mark.parametrize("dtype,head_dim,batches", [(BF16, 128, (100, 304, 650, 930)), (F16, 64, (300, 640, 1850)),
                                                    (F32, 128, (160, 320)), (BF16, 256, (160, 320))])
def test_decode_gives_the_bits_of_one_sequence_in_any_batch(dtype, head_dim, batches, longest):
    # a CTA a chunk, a pair or a share, as the batch grows: one sequence's bits stay
    for batch in batches:
        lens = [(longest * (1 + (7 * b) % 10)) // 10 for b in range(batch)]
        lens[batch // 3] = longest
        d = Decode(dtype, lens, 2, 1, head_dim, 16)
        out, lse = d.run()
        for b in (0, batch // 3, batch - 1):
            alone, alone_lse = d.run(q=d.q[b:b + 1].contiguous(), table=d.table[b:b + 1].contiguous(),
                                     lens=d.lens[b:b + 1].contiguous())
            assert torch.equal(alone[0], out[b]) and torch.equal(alone_lse[0], lse[b]), (batch, b)
        some = [0, batch // 3]
        want, _, tol, _ = ref.decode(d.q[some], d.k, d.v, d.table[some], [lens[b] for b in some], d.scale)
        ref.assert_near(out[some], want, tol, f"{batch} sequences")


def test_workspace_bytes_never_shrink_with_max_len():
    k = torch.empty((2, 16, 4, 64), dtype=BF16, device="cuda")
    cache = df.PagedCache(k, torch.empty_like(k))
    for batch in (1, 3, 76, 77, 114, 200, 1000):
        for heads in (4, 8, 80):
            sizes = [df.detfold_attn_decode_workspace_bytes(cache, batch, heads, n)
                     for n in list(range(0, 700, 13)) + [1 << x for x in range(10, 31)]]
            assert sizes == sorted(sizes), (batch, heads)


# ------------------------------------------------------------------ what the binding refuses

def test_binding_refusals_on_the_gpu():
    d = Decode(BF16, [40, 3], 8, 2, 64, 16)
    out = torch.empty_like(d.q)

    def call(**kw):
        a = dict(out=out, q=d.q, cache=d.cache, block_table=d.table, seq_lens=d.lens, max_len=d.max_len, scale=1.0)
        a.update(kw)
        df.detfold_attn_decode(**a)
    call()
    for kw in (dict(q=d.q.float()), dict(out=out.half()), dict(q=d.q.cpu()), dict(block_table=d.table.long()),
               dict(seq_lens=d.lens.long()), dict(q=None), dict(lse=torch.empty((2, 8), dtype=BF16, device="cuda")),
               dict(status=torch.zeros(1, device="cuda")), dict(max_len="40")):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=d.q[:1]), dict(q=d.q[:, :, :32]), dict(out=out.transpose(1, 2).contiguous().transpose(1, 2)),
               dict(block_table=d.table[:1]), dict(block_table=d.table[0]), dict(seq_lens=d.lens[:1]),
               dict(lse=torch.empty((2, 4), device="cuda")), dict(workspace=torch.empty(64, device="cuda")[::2])):
        with pytest.raises(ValueError):
            call(**kw)
    S = df.STATUS
    for kw, code in ((dict(max_len=1000), "DETFOLD_ERR_LEN"), (dict(window=-1), "DETFOLD_ERR_ARG"),
                     (dict(q=d.q[:, :7], out=out[:, :7]), "DETFOLD_ERR_ARG"), (dict(out=d.q), "DETFOLD_ERR_OVERLAP")):
        with pytest.raises(df.DetfoldError) as e:
            call(**kw)
        assert e.value.status == S[code], kw
    long = Decode(BF16, [4000], 8, 2, 64, 16)
    with pytest.raises(df.DetfoldError) as e:
        df.detfold_attn_decode(torch.empty_like(long.q), long.q, long.cache, long.table, long.lens, 4000, 1.0)
    assert e.value.status == S["DETFOLD_ERR_WORKSPACE"]

    a = Append(BF16, 6, 4, 2, 64, 64, False)
    q_out = torch.empty((6, 4, 64), dtype=BF16, device="cuda")

    def add(**kw):
        b = dict(cache=a.cache, k=a.nk, v=a.nv, slots=a.slots, rope=a.rope, positions=a.positions, q=a.q, q_out=q_out)
        b.update(kw)
        df.detfold_kv_append(**b)
    add()
    for kw in (dict(k=a.nk.float()), dict(slots=a.slots.int()), dict(positions=a.positions.int()), dict(q=a.q.half()),
               dict(v=a.nv.cpu())):
        with pytest.raises(TypeError):
            add(**kw)
    for kw in (dict(k=a.nk[:5]), dict(k=a.nk[:, :1]), dict(v=a.nv[:, :, :32]), dict(slots=a.slots[:5]), dict(positions=None),
               dict(q_out=None), dict(q=None), dict(q_out=q_out[:, :3])):
        with pytest.raises(ValueError):
            add(**kw)
    with pytest.raises(df.DetfoldError) as e:
        add(rope=df.Rope(torch.zeros((10, 128), device="cuda")))  # wider than the head
    assert e.value.status == S["DETFOLD_ERR_ARG"]
    with pytest.raises(df.DetfoldError) as e:
        add(k=a.k[0, :6])  # the cache's own rows
    assert e.value.status == S["DETFOLD_ERR_OVERLAP"]
    with pytest.raises(ValueError):
        df.PagedCache(a.k, a.v[:, :, :1])
    with pytest.raises(ValueError):
        df.PagedCache(a.k.transpose(2, 3), a.v.transpose(2, 3))
    with pytest.raises(TypeError):
        df.PagedCache(a.k, a.v.float())

    parts, lses = join_inputs(BF16, 3, (5,), 64)
    for bad in (dict(parts=[parts[0], parts[1], parts[2].float()]), dict(lses=[lses[0], lses[1], lses[2].half()])):
        with pytest.raises(TypeError):
            df.detfold_attn_join(**{**dict(out=torch.empty_like(parts[0]), parts=parts, lses=lses), **bad})
    with pytest.raises(ValueError):
        df.detfold_attn_join(torch.empty_like(parts[0]), parts, lses[:2])
    with pytest.raises(ValueError):
        df.detfold_attn_join(torch.empty((4, 64), dtype=BF16, device="cuda"), parts, lses)
    with pytest.raises(df.DetfoldError) as e:
        df.detfold_attn_join(torch.empty_like(parts[0]), [], [])
    assert e.value.status == S["DETFOLD_ERR_WORLD"]
    torch.cuda.synchronize()
