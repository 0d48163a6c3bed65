"""Attention of drafted trees on the GPU against 64 bits: types, head layouts, sizes where tiles,
chunks, pages and words end, masks that leave a row empty, and what masked places hold."""
import math

import pytest
import torch

import tree_ref as ref
from attn_ref import U, assert_near, final_round

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DEV = "cuda"


@pytest.fixture(scope="module")
def df():
    import deterministic_fixed_order_gb300 as m
    return m


class Case:
    """A cache with every sequence's tokens in pages of any order, the rest NaN."""

    def __init__(self, dtype, lens, nodes, hq, hk, d, page, counts=None, window=0, layout="token", seed=1, masks=None,
                 spare=2, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.nodes, self.window, self.page = lens, nodes, window, page
        self.counts = counts if counts is not None else [nodes] * len(lens)
        self.given = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
        batch = len(lens)
        self.max_len = max(n + max(0, min(c, nodes)) for n, c in zip(lens, self.counts))
        width = max(1, -(-self.max_len // page)) + 1
        used = [-(-(n + c) // page) for n, c in zip(lens, self.counts)]
        pages = sum(used) + spare
        order = torch.randperm(pages, generator=g).int()
        table = torch.full((batch, width), -7, dtype=torch.int32)
        shape = (pages, hk, page, d) if layout == "head" else (pages, page, hk, d)
        k, v = (torch.randn(shape, generator=g) for _ in range(2))
        if layout == "head":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        at = 0
        stale = torch.ones(pages, page, dtype=torch.bool)
        for b, u in enumerate(used):
            mine = order[at:at + u]
            first = max(0, lens[b] + 1 - window) // page if window else 0
            table[b, first:u] = mine[first:]
            n = lens[b] + self.counts[b]
            for j, e in enumerate(mine.tolist()):
                stale[e, :max(0, min(page, n - j * page))] = False
            at += u
        k[stale], v[stale] = math.nan, math.nan
        if masks is None:
            masks = [ref.words(ref.ancestors(ref.parents_of(seed * 100 + b, c)), nodes) for b, c in enumerate(self.counts)]
        self.mask = torch.stack(masks).to(DEV)
        self.q = torch.randn(batch, nodes, hq, d, generator=g).mul(1.5).to(dtype).to(DEV)
        self.k, self.v = (x.to(dtype).to(DEV) if layout == "token" else
                          x.transpose(1, 2).contiguous().to(dtype).to(DEV).transpose(1, 2) for x in (k, v))
        self.table = table.to(DEV)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.scale = d ** -0.5 if scale is None else scale

    def run(self, df, max_len=None, out=None, stream=None, status=None, extra=0):
        b, t, h, _ = self.q.shape
        max_len = self.max_len if max_len is None else max_len
        cache = df.PagedCache(self.k, self.v)
        need = df.detfold_attn_tree_workspace_bytes(cache, b, t, h, max_len)
        ws = torch.full((max(16, need + extra),), 0xff, dtype=torch.uint8, device=DEV)
        out = torch.full_like(self.q, 7) if out is None else out
        lse = torch.full((b, t, h), 7.0, device=DEV)
        df.detfold_attn_tree(out, self.q, cache, self.table, self.lens_t, self.mask, max_len, self.scale,
                             node_counts=self.given, window=self.window, lse=lse, workspace=ws, status=status,
                             stream=stream)
        return out, lse

    def want(self):
        return ref.attend(self.q, self.k, self.v, self.table, self.lens, self.mask, self.scale, self.counts, self.window)

    def check(self, df, **kw):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, lse = self.run(df, status=status, **kw)
        o, s, tol, ltol, live = self.want()
        assert int(status) == 0
        rows = live.to(DEV)
        assert_near(out[rows], o[live], tol[live], "out")
        assert_near(lse[rows], s[live], ltol[live], "lse")
        assert bool((out[~rows] == 7).all()) and bool((lse[~rows] == 7).all()), "rows behind the last node"
        return out, lse


# (lens, nodes, q_heads, kv_heads, head_dim, page)
SHAPES = [
    ([0], 1, 1, 1, 64, 16),
    ([1], 2, 4, 2, 64, 1),
    ([37], 7, 8, 8, 64, 16),
    ([63, 64, 65], 5, 6, 2, 128, 24),
    ([127, 128, 129, 0], 9, 8, 2, 128, 16),
    ([255, 256, 257], 33, 8, 2, 80, 32),
    ([300], 64, 8, 1, 128, 16),
    ([200, 3], 65, 4, 4, 96, 8),
    ([100], 130, 4, 2, 128, 64),
    ([50], 256, 8, 4, 64, 128),
    ([700, 10], 31, 14, 2, 256, 24),
    ([513], 26, 10, 2, 192, 16),
    ([1500], 17, 32, 4, 128, 16),
    ([2100, 900], 40, 16, 4, 128, 7),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_values(df, dtype, shape):
    Case(dtype, *shape).check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 72, 88, 104, 120, 136, 160, 176, 200, 216, 240, 248, 256])
def test_head_dims(df, dtype, d):
    Case(dtype, [70, 150], 11, 6, 2, d, 16, counts=[11, 4], seed=d).check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("page", [1, 5, 16, 128, 300])
def test_pages(df, dtype, layout, page):
    Case(dtype, [333, 0, 40], 20, 8, 2, 128, page, counts=[20, 7, 1], layout=layout, seed=page).check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("window", [12, 13, 64, 128, 129, 500, 5000])
def test_windows(df, dtype, window):
    Case(dtype, [0, 3, 64, 200, 1001], 12, 8, 4, 64, 16, counts=[12, 12, 5, 1, 9], window=window, seed=window).check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_counts_none_and_padding(df, dtype):
    Case(dtype, [100, 0, 50, 0, 9], 24, 4, 1, 128, 16, counts=[24, 0, 0, 3, 1]).check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("group", [1, 3, 8, 16, 20, 130])
def test_groups(df, dtype, group):
    Case(dtype, [90, 140], 5, 2 * group, 2, 64, 16, seed=group).check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_any_masks(df, dtype):
    """Bits that are no tree's, rows without any, bits behind the last node."""
    g = torch.Generator().manual_seed(5)
    nodes, masks = 100, []
    for b in range(3):
        m = torch.randint(-2 ** 63, 2 ** 63 - 1, (nodes, 2), generator=g)
        m[::7] = 0
        m[3] = -1
        masks.append(m)
    Case(dtype, [0, 5, 400], nodes, 4, 2, 128, 16, counts=[100, 70, 30], masks=masks).check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_rows_that_see_nothing(df, dtype):
    masks = [torch.zeros(6, 1, dtype=torch.int64) for _ in range(2)]
    masks[0][2] = 4
    out, lse = Case(dtype, [0, 0], 6, 4, 2, 64, 16, masks=masks).check(df)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n", [0, 50, 130])
def test_masked_places_may_hold_anything(df, dtype, d, value, n):
    """Drafted tokens that most nodes do not attend to hold NaN or infinities, in keys and values."""
    nodes = 40
    c = Case(dtype, [n], nodes, 8, 2, d, 16, masks=[ref.words(ref.ancestors(ref.parents_of(3, nodes, "roots")), nodes)])
    for i in (0, 7, 39):
        t = n + i
        at = int(c.table[0, t // 16]), t % 16
        c.v[at][:, ::5] = value
        if i == 7:
            c.k[at] = value
    out, lse = c.run(df)
    clean = torch.ones(nodes, dtype=torch.bool)
    clean[[0, 7, 39]] = False
    o, s, tol, ltol, _ = c.want()
    assert_near(out[0, clean.to(DEV)], o[0, clean], tol[0, clean], "out of nodes that do not attend to them")
    assert_near(lse[0, clean.to(DEV)], s[0, clean], ltol[0, clean], "lse")
    for i in (0, 39):  # those that do: the formula's value in each place
        got, want = out[0, i].double().cpu(), o[0, i]
        assert bool((torch.isnan(got) == torch.isnan(want)).all())
        assert bool((got[torch.isinf(want)] == want[torch.isinf(want)]).all())
        fine = torch.isfinite(want)
        assert bool(torch.isfinite(got[fine]).all())
    assert bool(torch.isnan(out[0, 7]).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("window", [0, 30])
def test_values_that_are_not_finite_in_committed_tokens(df, dtype, window):
    """An infinite value gives the infinity to the nodes that attend to it, and nothing to those whose
    window has passed it."""
    c = Case(dtype, [200], 20, 4, 2, 128, 16, window=window,
             masks=[ref.words(ref.ancestors(ref.parents_of(3, 20, "chain")), 20)])
    for t in ((171, 180, 199) if window else (5, 100, 199)):
        at = int(c.table[0, t // 16]), t % 16
        c.v[at][:, t % 7] = math.inf
    out, _ = c.run(df)
    want = c.want()[0][0]
    got = out[0].double().cpu()
    assert bool((torch.isinf(got) == torch.isinf(want)).all())
    assert bool((got[torch.isinf(want)] > 0).all())
    assert not bool(torch.isnan(got).any())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("gap", [0, 16, 24, 40, 60])
def test_infinite_values_of_small_weights(df, dtype, gap):
    """A token that every node attends to, whose score is up to 60 under the others': e^-60 of infinity is infinity."""
    c = Case(dtype, [700], 9, 4, 2, 64, 16, scale=1.0)
    c.q.zero_()[..., 0] = 1
    finite = ~torch.isnan(c.k[..., :1].float()).expand_as(c.k)
    c.k.copy_(torch.where(finite, 0.0, math.nan))
    for t, sign in ((3, 1), (300, -1), (530, 1)):
        at = int(c.table[0, t // 16]), t % 16
        c.k[at][:, 0] = -gap
        c.v[at][:, t % 64] = sign * math.inf
    got, want = c.run(df)[0][0].double().cpu(), c.want()[0][0]
    assert bool(torch.isinf(want).any()) and not bool(torch.isnan(got).any())
    assert bool((torch.where(torch.isinf(want), want, 0.0) == torch.where(torch.isinf(got), got, 0.0)).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("gap", [0, 8, 16])
@pytest.mark.parametrize("n", [0, 70, 500])
def test_infinite_values_of_small_weights_among_drafted_tokens(df, dtype, gap, n):
    """The same of drafted tokens, which some nodes attend to: the infinity for these, nothing for the others. Weights are held
    down to e^-22 of the largest there in float16."""
    nodes = 12
    sets = [{i} | ({3} if i % 3 == 0 else set()) | ({7} if i > 6 else set()) for i in range(nodes)]
    c = Case(dtype, [n], nodes, 4, 2, 64, 16, scale=1.0, masks=[ref.words(sets, nodes)])
    c.q.zero_()[..., 0] = 1
    finite = ~torch.isnan(c.k[..., :1].float()).expand_as(c.k)
    c.k.copy_(torch.where(finite, 0.0, math.nan))
    for j, sign in ((3, 1), (7, -1)):
        at = int(c.table[0, (n + j) // 16]), (n + j) % 16
        c.k[at][:, 0] = -gap
        c.v[at][:, 5 + j] = sign * math.inf
    got, want = c.run(df)[0][0].double().cpu(), c.want()[0][0]
    assert bool(torch.isinf(want).any()) and not bool(torch.isnan(got).any())
    assert bool((torch.where(torch.isinf(want), want, 0.0) == torch.where(torch.isinf(got), got, 0.0)).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_scores_of_all_sizes(df, dtype):
    """Maxima that jump from tile to tile, by little and by much, upwards and downwards."""
    c = Case(dtype, [1200], 16, 8, 2, 128, 16)
    g = torch.Generator().manual_seed(2)
    size = torch.exp(torch.randn(c.k.shape[0], generator=g) * 1.5).to(DEV).to(dtype)
    c.k.mul_(size[:, None, None, None])
    c.check(df)
    up = torch.arange(1216, device=DEV)
    at = (c.table[0].long()[up // 16], up % 16)
    q = c.q[0, 0, 0]
    for sign in (1, -1):
        c.k[at] = ((q.float() * sign * 0.02)[None, None] * (up[:, None, None] / 12.0)).to(dtype).expand(-1, 2, -1)
        c.check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("size", [1, -1])
def test_scores_that_are_large_and_close(df, dtype, size):
    """Scores of 2^14 and a few units: what a maximum loses by rounding would be the whole weight. The products are
    exact, so that a score's only error is its size's last places, four of them at most."""
    c = Case(dtype, [700, 3], 20, 4, 2, 64, 16, scale=1.0)
    c.q.zero_()[..., 0], c.q[..., 1] = 128, 1
    finite = ~torch.isnan(c.k[..., :1].float())
    steps = torch.arange(c.k.shape[0] * c.k.shape[1], device=DEV).reshape(c.k.shape[:2]) % 7
    c.k[..., 2:] = torch.where(finite, 0.0, math.nan).to(dtype)
    c.k[..., 0] = torch.where(finite[..., 0], 128.0 * size, math.nan).to(dtype)
    c.k[..., 1] = torch.where(finite[..., 0], steps[..., None].float(), math.nan).to(dtype)
    out, lse = c.run(df)
    o, s, _, _, _ = c.want()
    score = 4 * U * (2 ** 14 + 7)
    v = float(c.v[finite.expand_as(c.v)].double().abs().max())
    tol = 2 * v * (score + 8 * U + (720 + 64) * 2 * U + 2.0 ** -16)
    assert_near(out, o, tol + final_round(o, dtype), "out")
    assert_near(lse, s, torch.full_like(s, 2 * (score + 8 * U + (720 + 64) * 2 * U) + 8 * U * 2 ** 14), "lse")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_that_are_not_finite_in_many_sequences(df, dtype, d):
    """More sequences than run at once, each a few tokens long and with an infinite value that some of its nodes attend to:
    what one leaves behind must not reach the next."""
    nodes, batch = 6, 500
    mask = ref.words(ref.ancestors(ref.parents_of(3, nodes, "roots")), nodes)
    c = Case(dtype, [b % 9 for b in range(batch)], nodes, 2, 1, d, 16, masks=[mask] * batch)
    for b in range(batch):
        c.v[int(c.table[b, 0]), b % 9 + b % nodes, 0, b % d] = math.inf if b & 1 else -math.inf
    out, lse = c.run(df)
    o, s, tol, ltol, _ = c.want()
    odd = ~torch.isfinite(o)
    rest = torch.ones(batch, nodes, dtype=torch.bool)
    rest[torch.arange(batch), torch.arange(batch) % nodes] = False
    assert_near(out[rest.to(DEV)], o[rest], tol[rest], "nodes that do not attend to it")
    got = out.double().cpu()
    assert bool((torch.isinf(got) == odd).all()) and bool((got[odd] == o[odd]).all())
    assert_near(lse, s, ltol, "lse")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-6, 3.0])
def test_scales(df, dtype, scale):
    Case(dtype, [150], 10, 4, 2, 64, 16, scale=scale).check(df)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_strides_and_alignment(df, dtype):
    c = Case(dtype, [77, 300], 13, 6, 2, 64, 16)
    want = c.check(df)[0]
    b, t, h, d = c.q.shape
    whole = torch.randn(b, h, t, 3 * d + 1, device=DEV).to(dtype)
    odd = whole[..., 1:1 + d].transpose(1, 2)  # heads outside nodes, one element off
    odd.copy_(c.q)
    c.q = odd
    room = torch.zeros(t, b, h, d + 3, device=DEV, dtype=dtype)
    out = room[..., 3:].transpose(0, 1)
    c.run(df, out=out)
    assert torch.equal(out, want)
    assert bool((room[..., :3] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_the_same_bits_alone_and_in_any_batch(df, dtype):
    """A sequence's bits follow from itself: not from the batch, its pages, its padding or max_len."""
    lens, counts = [1900, 40, 0, 700, 2500, 129], [20, 3, 20, 11, 7, 20]
    masks = [ref.words(ref.ancestors(ref.parents_of(b, c)), 20) for b, c in enumerate(counts)]
    c = Case(dtype, lens, 20, 16, 2, 128, 16, counts=counts, masks=masks)
    out, lse = c.run(df)
    big = 40  # many of them: another way to share the work out
    for b, (n, k) in enumerate(zip(lens, counts)):
        one = Case(dtype, [n], k, 16, 2, 128, 16, masks=[masks[b][:k]])
        many = Case(dtype, [n] * big, 20, 16, 2, 128, 16, counts=[k] * big, masks=[masks[b]] * big)
        for other, rows in ((one, 1), (many, big)):
            t = torch.arange(n + k, device=DEV)
            for r in range(rows):
                to = (other.table[r].long()[t // 16], t % 16)
                at = (c.table[b].long()[t // 16], t % 16)
                other.k[to], other.v[to] = c.k[at], c.v[at]
            other.q[:, :k] = c.q[b, :k]
            for more in (0, 20000):
                if more:
                    pad = torch.full((rows, 2 * (n + more) // 16 + 2), -1, dtype=torch.int32, device=DEV)
                    pad[:, :other.table.shape[1]] = other.table
                    other.table = pad
                got, glse = other.run(df, max_len=other.max_len + more)
                for r in (0, rows - 1):
                    assert torch.equal(got[r, :k], out[b, :k]), (b, rows, more)
                    assert torch.equal(glse[r, :k], lse[b, :k])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_long(df, dtype):
    """Long enough that chunks are longer than the least and every CTA has several tiles."""
    Case(dtype, [30000], 8, 4, 1, 64, 16).check(df)


def test_offsets_past_32_bits(df):
    """A cache of more than 2^32 elements, the sequence's pages at its end."""
    pages, page, hk, d = 70000, 64, 8, 128
    if torch.cuda.mem_get_info()[0] < 22 * 2 ** 30:
        pytest.skip("needs 20 GB")
    k = torch.empty(pages, page, hk, d, dtype=BF16, device=DEV)
    v = torch.empty_like(k)
    g = torch.Generator(device=DEV).manual_seed(1)
    c = Case(BF16, [300], 10, 16, 8, 128, 64)
    used = -(-310 // 64)
    k[-used:] = torch.randn(used, page, hk, d, device=DEV, generator=g).to(BF16)
    v[-used:] = torch.randn(used, page, hk, d, device=DEV, generator=g).to(BF16)
    c.k, c.v = k, v
    c.table[0, :used] = torch.arange(pages - used, pages, device=DEV, dtype=torch.int32).flip(0)
    c.check(df)


# ------------------------------------------------------------------ what is refused, and indexes that are wrong

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("what", ["len", "negative", "count", "page", "negative page", "window page"])
def test_bad_indexes_give_nan(df, dtype, what):
    c = Case(dtype, [300, 700, 20], 9, 8, 2, 128, 16, counts=[9, 5, 9], window=100 if what == "window page" else 0)
    good = c.run(df)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    rows = 5
    if what == "len":
        c.lens_t[1] = c.max_len
    elif what == "negative":
        c.lens_t[1] = -1
    elif what == "count":
        c.given[1], rows = 10, 9
    elif what == "page":
        c.table[1, 3] = c.k.shape[0]
    elif what == "negative page":
        c.table[1, 43] = -1
    else:
        c.table[1, 40] = 1 << 30
    out, lse = c.run(df, status=status)
    assert int(status) == -8
    for b in (0, 2):
        assert torch.equal(out[b], good[0][b]) and torch.equal(lse[b], good[1][b])
    assert bool(torch.isnan(out[1, :rows]).all()) and bool(torch.isnan(lse[1, :rows]).all())
    assert bool((out[1, rows:] == 7).all())


def test_refusals(df):
    c = Case(BF16, [30], 8, 4, 2, 64, 16)
    cache = df.PagedCache(c.k, c.v)
    need = df.detfold_attn_tree_workspace_bytes(cache, 1, 8, 4, 3000)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    out, tree = torch.empty_like(c.q), df.tree
    table = torch.zeros(1, 200, dtype=torch.int32, device=DEV)

    def call(out=out, q=c.q, table=table, max_len=3000, workspace=ws, window=0, mask=c.mask):
        return tree.status_attn_tree(out, q, cache, table, c.lens_t, mask, max_len, 1.0, workspace=workspace,
                                     window=window)

    assert call(workspace=None) == -6 and call(workspace=ws[:-1]) == -6
    assert call(workspace=torch.empty(need + 8, dtype=torch.uint8, device=DEV)[8:]) == -6
    assert call(window=7) == -8 and call(max_len=3201) == -3 and call(out=c.q) == -5
    with pytest.raises(df.DetfoldError):
        df.detfold_attn_tree(c.q, c.q, cache, table, c.lens_t, c.mask, 3000, 1.0, workspace=ws)
    with pytest.raises(TypeError):
        call(mask=c.mask.int())
    with pytest.raises(ValueError):
        call(mask=c.mask[:, :7])
    with pytest.raises(TypeError):
        call(q=c.q.float())
    with pytest.raises(ValueError):
        tree.status_attn_tree(out, c.q, cache, table, c.lens_t.repeat(2), c.mask, 3000, 1.0)


def test_no_rows_is_a_no_op(df):
    c = Case(BF16, [30], 8, 4, 2, 64, 16)
    cache = df.PagedCache(c.k, c.v)
    for q, mask, lens, table in ((c.q[:0], c.mask[:0], c.lens_t[:0], c.table[:0]),
                                 (c.q[:, :0], c.mask[:, :0, :0], c.lens_t, c.table)):
        df.detfold_attn_tree(torch.empty_like(q), q, cache, table, lens, mask, 40, 1.0)


# ------------------------------------------------------------------ streams, graphs, threads

@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graphs_replay_with_new_inputs(df, dtype):
    """Two captured graphs with workspaces of their own, replayed on two streams at once."""
    cases = [Case(dtype, [1500, 300], 20, 8, 2, 128, 16, seed=s) for s in (1, 2)]
    made = []
    for c in cases:
        cache = df.PagedCache(c.k, c.v)
        need = df.detfold_attn_tree_workspace_bytes(cache, 2, 20, 8, c.max_len)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device=DEV)

        def call(c=c, cache=cache, ws=ws, out=out, lse=lse):
            df.detfold_attn_tree(out, c.q, cache, c.table, c.lens_t, c.mask, c.max_len, c.scale, lse=lse, workspace=ws)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
            call()
        made.append((c, g, out, lse, torch.cuda.Stream()))
    for again in range(3):
        for c, *_ in made:
            c.q.mul_(-0.9)
            c.lens_t[1] = 300 - again
            c.lens[1] = 300 - again
        torch.cuda.synchronize()
        for _ in range(3):
            for c, g, out, lse, stream in made:
                with torch.cuda.stream(stream):
                    g.replay()
        torch.cuda.synchronize()
        for c, g, out, lse, _ in made:
            want = c.run(df)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_calls_at_once(df, dtype):
    """Calls on several streams at a time, of sizes that share the GPU."""
    cases = [Case(dtype, [200 * s, 70], 10 + s, 8, 2, 128, 16, seed=s) for s in range(1, 6)]
    want = [c.run(df) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        got = [c.run(df, stream=None if i == 0 else None) for i, c in enumerate(cases)]
        torch.cuda.synchronize()
        outs = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                outs.append(c.run(df))
        torch.cuda.synchronize()
        for w, a, b in zip(want, got, outs):
            assert torch.equal(w[0], a[0]) and torch.equal(w[1], a[1])
            assert torch.equal(w[0], b[0]) and torch.equal(w[1], b[1])


def test_join_of_two_parts(df):
    """A rank with the first tokens alone and one with the rest and the tree: joined, the whole."""
    c = Case(F32, [320], 12, 8, 2, 64, 16)
    o, s, tol, ltol, _ = c.want()
    whole = c.run(df)
    cut = 160
    empty = torch.zeros_like(c.mask)
    cache = df.PagedCache(c.k, c.v)
    parts, lses = [], []
    for table, n, mask, counts in ((c.table[:, :11], cut, empty, torch.tensor([12], dtype=torch.int32, device=DEV)),
                                   (c.table[:, cut // 16:].contiguous(), 320 - cut, c.mask, None)):
        max_len = n + 12
        need = df.detfold_attn_tree_workspace_bytes(cache, 1, 12, 8, max_len)
        ws = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
        out, lse = torch.empty_like(c.q), torch.empty(1, 12, 8, device=DEV)
        df.detfold_attn_tree(out, c.q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), mask, max_len,
                             c.scale, node_counts=counts, lse=lse, workspace=ws)
        parts.append(out)
        lses.append(lse)
    out, lse = torch.empty_like(c.q), torch.empty(1, 12, 8, device=DEV)
    df.detfold_attn_join(out, parts, lses, lse=lse)
    # each part within its own bound, and the join's own few roundings
    assert_near(out, o, 3 * tol, "out")
    assert_near(lse, s, 3 * ltol, "lse")
    assert_near(whole[0], o, tol, "whole")
