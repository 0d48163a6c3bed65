"""The whole-number operators of a step with drafted tokens on the GPU, against plain Python: the
trees' layout, rows and pages that move, the bookkeeping of pages; then a whole step."""
import random

import pytest
import torch

import tree_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
I32 = {"dtype": torch.int32, "device": DEV}


@pytest.fixture(scope="module")
def df():
    import deterministic_fixed_order_gb300 as m
    return m


def ints(x):
    return torch.tensor(x, **I32)


# ------------------------------------------------------------------ plan

def plan(df, parents, lens, table, page, pages, counts=None, status=None):
    batch, nodes = len(parents), len(parents[0])
    mask = torch.full((batch, nodes, -(-nodes // 64)), 77, dtype=torch.int64, device=DEV)
    pos, slots = (torch.full((batch, nodes), 77, dtype=torch.int64, device=DEV) for _ in range(2))
    df.detfold_tree_plan(mask, ints(parents), ints(lens), ints(table), page, pages,
                         node_counts=None if counts is None else ints(counts), positions=pos, slots=slots, status=status)
    return mask.cpu(), pos.cpu(), slots.cpu()


@pytest.mark.parametrize("nodes", [1, 2, 31, 32, 33, 63, 64, 65, 128, 129, 192, 193, 255, 256])
@pytest.mark.parametrize("shape", ["tree", "chain", "roots"])
def test_plan(df, nodes, shape):
    r = random.Random(nodes)
    batch, page = 5, 16
    parents = [ref.parents_of(nodes + b, nodes, shape) for b in range(batch)]
    lens = [0, 1, 15, 16, 500]
    cols = (500 + nodes) // page + 1
    table = [[r.randrange(999) for _ in range(cols)] for _ in range(batch)]
    for counts in (None, [nodes, 0, 1, nodes // 2, nodes]):
        got = plan(df, parents, lens, table, page, 999, counts)
        for x, y in zip(got, ref.plan(parents, lens, table, page, 999, counts)):
            assert torch.equal(x, y)


def test_plan_of_bad_trees(df):
    parents = [[-1, 0, 1], [-1, 1, 0], [-2, 0, 0], [-1, 0, 3], [-1, 0, 1], [-1, 0, 1], [-1, 5, 1]]
    lens, counts = [5, 5, 5, 5, -1, 5, 5], [3, 3, 3, 3, 3, 4, 1]
    table = [[1, 2]] * 7
    status = torch.zeros(1, **I32)
    got = plan(df, parents, lens, table, 4, 9, counts, status)
    for x, y in zip(got, ref.plan(parents, lens, table, 4, 9, counts)):
        assert torch.equal(x, y)
    assert int(status) == -8
    status.zero_()
    got = plan(df, [[-1, 0, 1]], [7], [[1, 2]], 4, 9, status=status)  # past the table
    assert got[2].tolist() == [[11, -1, -1]] and int(status) == -8
    status.zero_()
    got = plan(df, [[-1, 0, 1]], [6], [[1, 9]], 4, 9, status=status)  # past the pool
    assert got[2].tolist() == [[-1, -1, -1]] and int(status) == -8


def test_plan_of_masks_alone(df):
    parents = ints([ref.parents_of(1, 50)])
    mask = torch.empty(1, 50, 1, dtype=torch.int64, device=DEV)
    df.detfold_tree_plan(mask, parents, ints([3]))
    assert torch.equal(mask.cpu()[0], ref.words(ref.ancestors(parents.tolist()[0]), 50))
    with pytest.raises(ValueError):
        df.detfold_tree_plan(mask, parents, ints([3]), slots=torch.empty(1, 50, dtype=torch.int64, device=DEV))
    df.detfold_tree_plan(mask[:0], parents[:0], ints([]))


# ------------------------------------------------------------------ rows and pages

def make_cache(dtype, pages, page, heads, d, layout, seed=1, offset=0):
    g = torch.Generator().manual_seed(seed)
    got = []
    for _ in range(2):
        shape = (pages, heads, page, d) if layout == "head" else (pages, page, heads, d)
        x = torch.randn(shape, generator=g).to(dtype)
        flat = torch.zeros(x.numel() + offset, dtype=dtype)
        flat[offset:] = x.flatten()
        x = flat.to(DEV)[offset:].view(shape)
        got.append(x.transpose(1, 2) if layout == "head" else x)
    return got


CACHES = [(torch.bfloat16, 16, 8, 128, "token", 0), (torch.float16, 8, 2, 64, "head", 0), (torch.float32, 5, 3, 80, "token", 0),
          (torch.bfloat16, 1, 1, 8, "token", 0), (torch.bfloat16, 4, 2, 33, "head", 0), (torch.float16, 16, 4, 64, "token", 1),
          (torch.float32, 32, 1, 6, "head", 1), (torch.bfloat16, 7, 20, 256, "head", 4)]


@pytest.mark.parametrize("dtype,page,heads,d,layout,offset", CACHES)
def test_compact(df, dtype, page, heads, d, layout, offset):
    r = random.Random(page * d)
    nodes, batch = 256, 9
    lens = [0, 1, page - 1, page, 3 * page + 1, 40, 7, 2, 5]
    cols = (max(lens) + nodes) // page + 1
    pages = cols * batch
    k, v = make_cache(dtype, pages, page, heads, d, layout, offset=offset)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3))[:cols * batch].view(batch, cols).int()
    paths = [[0], [0, 1, 2], [1], sorted(r.sample(range(nodes), 17)), list(range(1, 201)), [0, 2, 3, 4, 9, 10, 100, 255],
             [], list(range(nodes)), sorted(r.sample(range(nodes), 8))]
    path = ints([p + [-5] * (nodes - len(p)) for p in paths])
    want_k, want_v = k.clone(), v.clone()
    for b, p in enumerate(paths):
        for i, j in enumerate(p):
            at = [(int(table[b, t // page]), t % page) for t in (lens[b] + i, lens[b] + j)]
            want_k[at[0]], want_v[at[0]] = k[at[1]], v[at[1]]
    status = torch.zeros(1, **I32)
    df.detfold_kv_compact(df.PagedCache(k, v), table.to(DEV), ints(lens), path, ints([len(p) for p in paths]), status=status)
    assert torch.equal(k, want_k) and torch.equal(v, want_v) and int(status) == 0


def test_compact_leaves_bad_sequences(df):
    k, v = make_cache(torch.bfloat16, 40, 4, 2, 64, "token")
    before = k.clone(), v.clone()
    table = torch.arange(40).view(8, 5).int()
    table[5, 4], table[6, 0] = 40, -1
    paths = [[0, 2, 2], [3, 1, 0], [0, 256, 300], [-1, 2, 3], [0, 2, 4], [9, 10, 11], [1, 2, 3], [0, 5, 19]]
    lens, counts = [4, 4, 4, 4, -1, 8, 0, 4], [3, 3, 2, 3, 3, 3, 3, 3]
    for b in range(8):
        status = torch.zeros(1, **I32)
        df.detfold_kv_compact(df.PagedCache(k, v), table[b:b + 1].to(DEV), ints(lens[b:b + 1]), ints(paths[b:b + 1]),
                              ints(counts[b:b + 1]), status=status)
        assert int(status) == -8, b
        assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    for n in (-1, 4):
        status = torch.zeros(1, **I32)
        df.detfold_kv_compact(df.PagedCache(k, v), table[:1].to(DEV), ints([4]), ints([[1, 2, 3]]), ints([n]), status=status)
        assert int(status) == -8 and torch.equal(k, before[0])


@pytest.mark.parametrize("dtype,page,heads,d,layout,offset", CACHES)
@pytest.mark.parametrize("count", [1, 3, 150])
@pytest.mark.parametrize("partial", [False, True])
def test_copy_pages(df, dtype, page, heads, d, layout, offset, count, partial):
    r = random.Random(count)
    pages = 2 * count + 5
    k, v = make_cache(dtype, pages, page, heads, d, layout, offset=offset)
    order = r.sample(range(pages), 2 * count)
    src, dst = order[:count], order[count:]
    rows = [r.randint(0, page) for _ in src]
    if count > 2:
        src[1], dst[2] = -1, -3
    want_k, want_v = k.clone(), v.clone()
    for a, b, n in zip(src, dst, rows):
        if a >= 0 and b >= 0:
            n = n if partial else page
            want_k[b, :n], want_v[b, :n] = k[a, :n], v[a, :n]
    df.detfold_kv_copy_pages(df.PagedCache(k, v), ints(src), ints(dst), rows=ints(rows) if partial else None)
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_copy_pages_of_one_buffer_and_bad_pairs(df):
    both = torch.randn(12, 2, 16, 4, 64, device=DEV).bfloat16()  # a page's keys, then its values
    k, v = both[:, 0], both[:, 1]
    want = both.clone()
    want[7], want[3] = both[2], both[11]
    status = torch.zeros(1, **I32)
    df.detfold_kv_copy_pages(df.PagedCache(k, v), ints([2, 11, 5, 12, 1, 4]), ints([7, 3, 5, 0, 12, -1]), status=status)
    assert torch.equal(both, want) and int(status) == -8
    for bad in (-1, 17):
        status.zero_()
        df.detfold_kv_copy_pages(df.PagedCache(k, v), ints([2]), ints([8]), rows=ints([bad]), status=status)
        assert torch.equal(both, want) and int(status) == -8
    df.detfold_kv_copy_pages(df.PagedCache(k, v), ints([]), ints([]))


# ------------------------------------------------------------------ the pool

def step(df, refs, table, lens, origin, keep, want, page, cols, in_place=False, status=None):
    n, m = len(lens), len(origin)
    a = ints(refs)
    out = a if in_place else torch.full_like(a, 99)
    to = torch.full((m, cols + 3), 99, **I32)[:, :cols]
    rest = [torch.full((m,), 99, **I32) for _ in range(4)]
    t = ints(table).view(n, cols) if n else torch.empty(0, cols, **I32)
    status = torch.zeros(1, **I32) if status is None else status
    df.detfold_pages_step(out, to, *rest, a, t, ints(lens), ints(origin), ints(keep), ints(want), page, status=status)
    return [out.tolist(), to.tolist()] + [x.tolist() for x in rest] + [int(status)]


def check_step(df, refs, table, lens, origin, keep, want, page, cols):
    w = ref.pages_step(refs, table, lens, origin, keep, want, page, cols)
    for in_place in (False, True):
        got = step(df, refs, table, lens, origin, keep, want, page, cols, in_place)
        for what, x, y in zip(("refs", "table", "lens", "src", "dst", "rows"), got, w):
            assert x == y, what
        assert got[6] in {0: (0,), 1: (-8,), 2: (-9,), 3: (-8, -9)}[w[6]]
    return w


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("page", [1, 4, 16])
def test_pages_over_many_steps(df, seed, page):
    """A pool lived in: begin, grow, cut back, fork, end, with shared prompts and with too few pages."""
    r = random.Random(seed * 31 + page)
    cols, pool = r.choice([3, 9, 40]), r.choice([20, 200, 5000])
    refs = [0] * pool
    for i in r.sample(range(pool), pool // 10):
        refs[i] = 1  # something else holds them
    table, lens = [], []
    for _ in range(12):
        m = r.choice([0, 1, 3, 10, 33])
        origin, keep, want = [], [], []
        for b in range(m):
            o = r.choice([-1, b if b < len(lens) else -1, r.randrange(len(lens)) if lens else -1])
            k = 0 if o < 0 else r.choice([lens[o], lens[o], r.randint(0, lens[o])])
            origin.append(o)
            keep.append(k)
            want.append(min(cols * page, k + r.choice([0, 1, page, r.randint(0, 3 * page)])))
        refs, table, lens, src, dst, rows, _ = check_step(df, refs, table, lens, origin, keep, want, page, cols)
        # what a row may write to is its own
        for t, n, k in zip(table, lens, keep):
            assert all(refs[e] == 1 for e in t[k // page:-(-n // page)] if n > k)
        held = [e for t, n in zip(table, lens) for e in t[:-(-n // page)]]
        assert all(refs[e] >= held.count(e) for e in set(held))


def test_pages_of_large_pools(df):
    r = random.Random(9)
    for rows, pool, cols in ((4096, 30000, 6), (1, 100001, 3000), (700, 65536, 90)):
        refs = [int(r.random() < 0.2) for _ in range(pool)]
        free = [i for i, x in enumerate(refs) if x == 0]
        r.shuffle(free)
        page, lens, table = 8, [], []
        for _ in range(rows):
            n = r.randint(0, min(cols, len(free) // rows) * page)
            mine = [free.pop() for _ in range(-(-n // page))]
            for e in mine:
                refs[e] = 1
            lens.append(n)
            table.append(mine + [-1] * (cols - len(mine)))
        origin = [b if r.random() < 0.6 else r.randrange(rows) for b in range(rows)]
        keep = [lens[o] if r.random() < 0.7 else r.randint(0, lens[o]) for o in origin]
        want = [min(cols * page, k + r.randint(0, 20)) for k in keep]
        check_step(df, refs, table, lens, origin, keep, want, page, cols)


def test_pages_of_bad_rows(df):
    refs, table, lens = [1, 1, 2, 0, 0, 0], [[0, 1, 2], [2, 9, -1], [2, 4, 4]], [9, 8, 99]
    good = ([0, 1], [9, 0], [10, 0])
    for origin, keep, want in (good, ([3, 0], [0, 9], [0, 9]), ([-2, 0], [0, 9], [3, 9]), ([-1, 0], [1, 9], [3, 9]),
                               ([0, 0], [10, 9], [12, 9]), ([0, 0], [9, 9], [8, 9]), ([0, 0], [9, 9], [13, 9]),
                               ([2, 0], [4, 9], [4, 9]), ([1, 0], [7, -1], [8, 9])):
        check_step(df, refs, table, lens, origin, keep, want, 4, 3)


def test_pages_refusals(df):
    a = torch.zeros(8, **I32)
    t = torch.full((2, 3), -1, **I32)
    row = [torch.zeros(2, **I32) for _ in range(8)]
    with pytest.raises(df.DetfoldError):  # the new table is the old one
        df.detfold_pages_step(a, t, *row[:4], a, t, *row[4:], 4)
    with pytest.raises(ValueError):
        df.detfold_pages_step(a, t.clone(), *row[:4], a[:7], t, *row[4:], 4)
    with pytest.raises(df.DetfoldError):
        df.detfold_pages_step(a, t.clone(), *row[:4], a, t, *row[4:], 0)
    with pytest.raises(df.DetfoldError):
        df.detfold_pages_step(a, t.clone(), row[0], row[0], row[2], row[3], a, t, *row[4:], 4)


# ------------------------------------------------------------------ a whole step

def test_drafted_step_like_tokens_one_by_one(df):
    """Tokens drafted as a tree, laid out, appended, attended to; the accepted path kept; then the
    next token's attention: as if the path's tokens had been appended one by one."""
    hq, hk, d, page, nodes, batch = 8, 2, 64, 8, 20, 3
    g = torch.Generator(device=DEV).manual_seed(4)
    lens0, cols, pool = [0, 13, 40], 12, 60

    def rand(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    refs = torch.zeros(pool, **I32)
    table = torch.full((batch, cols), -1, **I32)
    lens = ints([0] * batch)

    def resize(origin, keep, want):
        nonlocal refs, table, lens
        m = len(origin)
        to, rest = torch.empty(m, cols, **I32), [torch.empty(m, **I32) for _ in range(4)]
        df.detfold_pages_step(refs, to, *rest, refs, table, lens, ints(origin), ints(keep), ints(want), page)
        table, lens = to, rest[0]
        df.detfold_kv_copy_pages(cache, rest[1], rest[2], rows=rest[3])

    cache = df.PagedCache(*(torch.full((pool, page, hk, d), float("nan"), device=DEV) for _ in range(2)))
    plain = df.PagedCache(*(torch.full((pool, page, hk, d), float("nan"), device=DEV) for _ in range(2)))
    angle = torch.arange(200, device=DEV, dtype=torch.float64)[:, None] * torch.logspace(0, -3, d // 2, device=DEV, dtype=torch.float64)
    rope = df.Rope(torch.cat([angle.cos(), angle.sin()], 1).float())
    resize([-1] * batch, [0] * batch, [n + nodes for n in lens0])
    own = torch.arange(batch * cols, **I32).view(batch, cols)  # the other cache's pages
    for b, n in enumerate(lens0):
        t = torch.arange(n, device=DEV)
        k, v = rand(n, hk, d), rand(n, hk, d)
        df.detfold_kv_append(cache, k, v, table[b].long()[t // page] * page + t % page, rope=rope, positions=t)
        df.detfold_kv_append(plain, k, v, own[b].long()[t // page] * page + t % page, rope=rope, positions=t)
    parents = [ref.parents_of(b, nodes) for b in range(batch)]
    mask = torch.empty(batch, nodes, 1, dtype=torch.int64, device=DEV)
    positions, slots = (torch.empty(batch, nodes, dtype=torch.int64, device=DEV) for _ in range(2))
    seq = ints(lens0)
    df.detfold_tree_plan(mask, ints(parents), seq, table, page, pool, positions=positions, slots=slots)
    k, v, q = rand(batch, nodes, hk, d), rand(batch, nodes, hk, d), rand(batch, nodes, hq, d)
    turned = torch.empty_like(q)
    df.detfold_kv_append(cache, k.view(-1, hk, d), v.view(-1, hk, d), slots.view(-1), rope=rope,
                         positions=positions.view(-1), q=q.view(-1, hq, d), q_out=turned.view(-1, hq, d))
    max_len = max(lens0) + nodes

    def workspace(n):
        return torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)

    out = torch.empty_like(q)
    df.detfold_attn_tree(out, turned, cache, table, seq, mask, max_len, d ** -0.5,
                         workspace=workspace(df.detfold_attn_tree_workspace_bytes(cache, batch, nodes, hq, max_len)))
    # the deepest node's path is accepted
    sets = [ref.ancestors(p) for p in parents]
    paths = [sorted(max(s, key=len)) for s in sets]
    longest = max(len(p) for p in paths)
    df.detfold_kv_compact(cache, table, seq, ints([p + [-1] * (longest - len(p)) for p in paths]), ints([len(p) for p in paths]))
    kept = [n + len(p) for n, p in zip(lens0, paths)]
    resize(list(range(batch)), kept, [n + 1 for n in kept])
    u = 2.0 ** -24
    one = torch.empty(1, hq, d, device=DEV)
    for b, p in enumerate(paths):
        for i, j in enumerate(p):
            at = torch.tensor([lens0[b] + i], device=DEV)
            slot = own[b].long()[at // page] * page + at % page
            got = torch.empty(1, hq, d, device=DEV)
            df.detfold_kv_append(plain, k[b, j:j + 1], v[b, j:j + 1], slot, rope=rope, positions=at, q=q[b, j:j + 1], q_out=got)
            n = int(at) + 1
            df.detfold_attn_decode(one, got, plain, own[b:b + 1], ints([n]), n, d ** -0.5,
                                   workspace=workspace(df.detfold_attn_decode_workspace_bytes(plain, 1, hq, n)))
            # each within its bound of the same value: scores of 64 products up to 40 in all, values up to 5
            assert float((one - out[b, j]).abs().max()) < 2 * 2 * 5 * (68 * 2 * u * 40 + (n + 72) * 2 * u)
        t = torch.arange(kept[b], device=DEV)
        x, y = (c.long()[t // page] for c in (table[b], own[b]))
        assert torch.equal(cache.k[x, t % page], plain.k[y, t % page])
        assert torch.equal(cache.v[x, t % page], plain.v[y, t % page])
    # two go on from the first, one from the third: forked, then each with a token of its own
    resize([0, 0, 2], [kept[0], kept[0], kept[2]], [kept[0] + 1, kept[0] + 1, kept[2] + 1])
    assert sorted(refs.tolist())[-1] == (2 if kept[0] >= page else 1)
    n = kept[0]
    slots = torch.stack([table[b].long()[n // page] * page + n % page for b in (0, 1)])
    assert slots[0] != slots[1]
    df.detfold_kv_append(cache, rand(2, hk, d), rand(2, hk, d), slots)
    t = torch.arange(n, device=DEV)
    for b in (0, 1):
        assert torch.equal(cache.k[table[b].long()[t // page], t % page], plain.k[own[0].long()[t // page], t % page])
