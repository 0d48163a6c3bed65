"""The operators of a step with drafted tokens as a server runs them: captured into graphs and replayed with
new inputs, on several streams at once, over caches past 32 bits, in very large batches."""
import random

import pytest
import torch

import tree_ref as ref
from test_gpu_tree import BF16, DEV, F16, F32, Case, df  # noqa: F401  (df: the fixture)
from test_gpu_tree_rows import check_step

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)


class Step:
    """Buffers of fixed sizes for one whole step: plan, attention, accepted paths, pages, copies."""

    def __init__(self, batch=6, nodes=24, hq=8, hk=2, d=64, page=8, cols=24, max_len=150, dtype=BF16):
        self.batch, self.nodes, self.page, self.max_len = batch, nodes, page, max_len
        self.pool, self.cols, self.d = batch * cols + 40, cols, d
        self.k, self.v = (torch.empty(self.pool, page, hk, d, dtype=dtype, device=DEV) for _ in range(2))
        self.q = torch.empty(batch, nodes, hq, d, dtype=dtype, device=DEV)
        self.out = torch.empty_like(self.q)
        self.lse = torch.empty(batch, nodes, hq, device=DEV)
        self.parents = torch.empty(batch, nodes, **I32)
        self.mask = torch.empty(batch, nodes, 1, dtype=torch.int64, device=DEV)
        self.positions, self.slots = (torch.empty(batch, nodes, dtype=torch.int64, device=DEV) for _ in range(2))
        self.table, self.new_table = (torch.empty(batch, cols, **I32) for _ in range(2))
        self.path = torch.empty(batch, 5, **I32)
        self.refs = torch.empty(self.pool, **I32)
        self.lens, self.counts, self.path_lens, self.held, self.origin, self.keep, self.room = (torch.empty(batch, **I32) for _ in range(7))
        self.new = [torch.empty(batch, **I32) for _ in range(4)]
        self.status = torch.zeros(1, **I32)

    def fill(self, seed):
        r, g = random.Random(seed), torch.Generator().manual_seed(seed)

        def put(to, x):
            to.copy_(torch.as_tensor(x).to(to.dtype))

        lens = [r.randint(0, self.max_len - self.nodes) for _ in range(self.batch)]
        counts = [r.randint(5, self.nodes) for _ in range(self.batch)]
        order = torch.randperm(self.pool, generator=g).int()[:self.batch * self.cols].view(self.batch, self.cols)
        used = [-(-(n + c) // self.page) for n, c in zip(lens, counts)]
        refs = torch.zeros(self.pool)
        for b, u in enumerate(used):
            refs[order[b, :u].long()] = 1
            order[b, u:] = -1
        put(self.k, torch.randn(self.k.shape, generator=g)), put(self.v, torch.randn(self.v.shape, generator=g))
        put(self.q, torch.randn(self.q.shape, generator=g))
        put(self.parents, [ref.parents_of(seed + b, self.nodes) for b in range(self.batch)])
        put(self.lens, lens), put(self.counts, counts), put(self.table, order), put(self.refs, refs)
        paths = [sorted(r.sample(range(c), 5)) for c in counts]
        sizes = [r.randint(1, 5) for _ in counts]
        put(self.path, paths), put(self.path_lens, sizes)
        put(self.held, [n + c for n, c in zip(lens, counts)])
        origin = [r.choice([b, r.randrange(self.batch)]) for b in range(self.batch)]
        put(self.origin, origin), put(self.keep, [lens[o] + sizes[o] for o in origin])
        put(self.room, [min(lens[o] + sizes[o] + r.randint(1, 2 * self.page), self.cols * self.page) for o in origin])

    def prepare(self, df):
        self.cache = df.PagedCache(self.k, self.v)
        need = df.detfold_attn_tree_workspace_bytes(self.cache, self.batch, self.nodes, self.q.shape[2], self.max_len)
        self.workspace = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)

    def run(self, df, stream=None):
        s = dict(status=self.status, stream=stream)
        df.detfold_tree_plan(self.mask, self.parents, self.lens, self.table, self.page, self.pool, node_counts=self.counts,
                             positions=self.positions, slots=self.slots, **s)
        df.detfold_attn_tree(self.out, self.q, self.cache, self.table, self.lens, self.mask, self.max_len, self.d ** -0.5,
                             node_counts=self.counts, lse=self.lse, workspace=self.workspace, **s)
        df.detfold_kv_compact(self.cache, self.table, self.lens, self.path, self.path_lens, **s)
        df.detfold_pages_step(self.refs, self.new_table, *self.new, self.refs, self.table, self.held, self.origin, self.keep,
                              self.room, self.page, **s)
        df.detfold_kv_copy_pages(self.cache, self.new[1], self.new[2], rows=self.new[3], **s)

    def results(self):
        return [x.clone() for x in (self.mask, self.positions, self.slots, self.out, self.lse, self.k, self.v, self.refs, self.new_table, *self.new, self.status)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def wanted(df, seed, **sizes):
    s = Step(**sizes)
    s.prepare(df)
    s.fill(seed), s.out.fill_(7), s.lse.fill_(7)
    s.run(df)
    torch.cuda.synchronize()
    return s.results()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_step_captured_and_replayed(df, dtype):
    """One graph of the whole step, replayed with other trees, lengths, pages and paths, on another stream than the
    capture's."""
    s = Step(dtype=dtype)
    s.prepare(df)
    s.fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run(df)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.run(df)
    for seed in (2, 3, 4):
        s.fill(seed), s.out.fill_(7), s.lse.fill_(7)
        s.workspace.fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        assert same(s.results(), wanted(df, seed, dtype=dtype)), seed
        assert int(s.status) == 0


def test_graphs_that_share_a_workspace(df):
    """Two graphs captured with one workspace, replayed one after the other."""
    a, b = Step(max_len=600, cols=80), Step(max_len=600, cols=80, nodes=9)
    a.prepare(df), b.prepare(df)
    a.workspace = b.workspace = max(a.workspace, b.workspace, key=len)
    graphs = []
    for s in (a, b):
        s.fill(1)
        s.run(df)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.run(df)
    for seed in (5, 6):
        for s in (a, b):
            s.fill(seed), s.out.fill_(7), s.lse.fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert same(a.results(), wanted(df, seed, max_len=600, cols=80))
        assert same(b.results(), wanted(df, seed, max_len=600, cols=80, nodes=9))


def test_steps_on_streams_at_once(df):
    """Steps of their own buffers on four streams, several times over, and through a raw handle."""
    steps = [Step() for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        s.prepare(df)
    for turn in range(3):
        for i, s in enumerate(steps):
            s.fill(10 * turn + i), s.out.fill_(7), s.lse.fill_(7)
        torch.cuda.synchronize()
        for s, stream in zip(steps, streams):
            s.run(df, stream=stream if turn else stream.cuda_stream)
        torch.cuda.synchronize()
        for i, s in enumerate(steps):
            assert same(s.results(), wanted(df, 10 * turn + i)), (turn, i)


def test_rows_and_pages_past_32_bits(df):
    """Caches of more than 2^32 bytes and elements: rows and pages at both ends."""
    page, heads, d = 16, 8, 128
    pages = (1 << 32) // (page * heads * d) + 3  # 2^32 elements and three pages
    k, v = (torch.empty(pages, page, heads, d, dtype=BF16, device=DEV) for _ in range(2))
    cache, last = df.PagedCache(k, v), pages - 1
    g = torch.Generator(device=DEV).manual_seed(3)
    for e in (0, 1, last - 1, last):
        for x in (k, v):
            x[e] = torch.randn(page, heads, d, device=DEV, generator=g).to(BF16)
    was = {e: (k[e].clone(), v[e].clone()) for e in (0, 1, last - 1, last)}
    table = torch.tensor([[last, 0]], **I32)
    one = dict(status=torch.zeros(1, **I32))
    df.detfold_kv_compact(cache, table, torch.tensor([14], **I32), torch.tensor([[1, 2, 5]], **I32), torch.tensor([3], **I32), **one)
    for i, x in enumerate((k, v)):
        assert torch.equal(x[last, 14], was[last][i][15]) and torch.equal(x[last, 15], was[0][i][0])
        assert torch.equal(x[0, 0], was[0][i][3]) and torch.equal(x[0, 1:], was[0][i][1:])
        assert torch.equal(x[last, :14], was[last][i][:14])
    df.detfold_kv_copy_pages(cache, torch.tensor([last - 1, 1], **I32), torch.tensor([0, last], **I32),
                             rows=torch.tensor([16, 9], **I32), **one)
    for i, x in enumerate((k, v)):
        assert torch.equal(x[0], was[last - 1][i]) and torch.equal(x[last, :9], was[1][i][:9])
        assert torch.equal(x[last, 9:14], was[last][i][9:14]) and torch.equal(x[1], was[1][i])
    assert int(one["status"]) == 0


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_very_many_sequences(df, dtype):
    """Thousands of sequences of every length up to 70, some without nodes: each as it is alone."""
    batch, nodes = 5000, 5
    counts = [b % 6 for b in range(batch)]
    masks = [ref.words(ref.ancestors(ref.parents_of(c, c) if c else []), nodes) if c else torch.zeros(nodes, 1, dtype=torch.int64) for c in range(6)]
    masks = [torch.cat([m, torch.zeros(nodes - m.shape[0], 1, dtype=torch.int64)]) for m in masks]
    c = Case(dtype, [b * 7 % 71 for b in range(batch)], nodes, 4, 2, 64, 16, counts=counts, masks=[masks[k] for k in counts])
    out, lse = c.run(df)
    cache = df.PagedCache(c.k, c.v)
    for b in random.Random(1).sample(range(batch), 40) + [0, batch - 1]:
        n = counts[b]
        one, sum_ = torch.full_like(c.q[b:b + 1], 7), torch.full((1, nodes, 4), 7.0, device=DEV)
        df.detfold_attn_tree(one, c.q[b:b + 1], cache, c.table[b:b + 1], c.lens_t[b:b + 1], c.mask[b:b + 1], 80, c.scale,
                             node_counts=c.given[b:b + 1], lse=sum_)
        assert torch.equal(out[b], one[0]) and torch.equal(lse[b], sum_[0]), b
        assert bool((out[b, n:] == 7).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_queries_that_sequences_share(df, dtype):
    """Queries broadcast over the batch and over heads (strides of 0) are only read."""
    c = Case(dtype, [90, 3, 40], 12, 8, 2, 128, 16)
    c.q = c.q[:1, :, :1].expand(3, 12, 8, 128)
    out, lse = c.run(df, out=torch.empty(3, 12, 8, 128, dtype=dtype, device=DEV))
    c.q = c.q.contiguous()
    want, sums = c.run(df)
    assert torch.equal(out, want) and torch.equal(lse, sums)


def test_no_status_word_and_no_lse(df):
    """Everything optional left out, with indexes that are out of range: no fault, the others' results as ever."""
    c = Case(BF16, [40, 60], 6, 4, 2, 64, 16)
    good = c.run(df)[0]
    cache, out = df.PagedCache(c.k, c.v), torch.zeros_like(c.q)
    c.table[1, 0] = 1 << 30
    df.detfold_attn_tree(out, c.q, cache, c.table, c.lens_t, c.mask, c.max_len, c.scale)
    assert torch.equal(out[0], good[0]) and bool(torch.isnan(out[1]).all())
    before = c.k.clone()
    df.detfold_kv_compact(cache, c.table[1:], torch.tensor([0], **I32), torch.tensor([[1]], **I32), torch.tensor([1], **I32))
    df.detfold_kv_copy_pages(cache, torch.tensor([1 << 30], **I32), torch.tensor([0], **I32))
    assert torch.equal(c.k.nan_to_num(), before.nan_to_num())


@pytest.mark.parametrize("pool", [524288, 524289, 700001])
def test_pages_of_very_large_pools(df, pool):
    """Pools that are looked through in tiles, nearly full, with enough free pages and with too few."""
    r = random.Random(pool)
    page, cols, rows = 16, 9, 300
    refs = [1] * pool
    for e in r.sample(range(pool), 2500):
        refs[e] = 0
    free = [e for e, x in enumerate(refs) if x == 0]
    r.shuffle(free)
    table, lens = [], []
    for _ in range(rows):
        n = r.randint(0, 3 * page)
        mine = [free.pop() for _ in range(-(-n // page))]
        for e in mine:
            refs[e] = 1
        table.append(mine + [-1] * (cols - len(mine)))
        lens.append(n)
    for more in (20, 100):
        origin = [r.choice([b, r.randrange(rows)]) for b in range(rows)]
        keep = [lens[o] for o in origin]
        check_step(df, refs, table, lens, origin, keep, [min(cols * page, k + r.randint(0, more)) for k in keep], page, cols)


def test_forks_of_one_sequence(df):
    """One prompt, as many rows as there may be, each of which goes on writing behind a page that they share."""
    page, cols, pool = 16, 40, 6000
    refs = [0] * pool
    mine = random.Random(2).sample(range(pool), 38)
    for e in mine:
        refs[e] = 1
    for length in (37 * 16 + 5, 38 * 16):
        check_step(df, refs, [mine + [-1, -1]], [length], [0] * 4096, [length] * 4096, [length + 1] * 4096, page, cols)
