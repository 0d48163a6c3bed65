"""Measured cases of the operators of a step with drafted tokens: laying out the
trees of drafted tokens, attention of their nodes over the paged cache, keeping
the accepted path's rows of the cache, copying pages, and the bookkeeping of
which sequence holds which pages (growing, forking, cutting back, freeing).

Each operator is given twice: in plain form (elementary torch operations in 32
bits, rounded once at the end) and, where ``own`` is true, as the calls that a
user makes of this package. ``exact`` computes the same from the definitions in
64 bits, where an operator computes with numbers or moves them.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WIDTH = {"f32": 4, "bf16": 2, "f16": 2}
NEG = float("-inf")


# ------------------------------------------------------------------ cases

def _attend(name, dtype, batch, nodes, q_heads, kv_heads, head_dim, page, max_len, lens="full", window=0,
            layout="token", ragged=False, mix=1):
    return {"name": name, "op": "attend", "dtype": dtype, "batch": batch, "nodes": nodes, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "max_len": max_len, "lens": lens,
            "window": window, "layout": layout, "ragged": ragged, "mix": mix}


def _plan(name, batch, nodes, page, max_len, shape="tree", mix=1):
    return {"name": name, "op": "plan", "batch": batch, "nodes": nodes, "page": page, "max_len": max_len,
            "shape": shape, "mix": mix}


def _compact(name, dtype, batch, nodes, path, kv_heads, head_dim, page, layout="token", mix=1):
    return {"name": name, "op": "compact", "dtype": dtype, "batch": batch, "nodes": nodes, "path": path,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "layout": layout, "mix": mix}


def _copy(name, dtype, pairs, kv_heads, head_dim, page, partial=False, layout="token", mix=1):
    return {"name": name, "op": "copy", "dtype": dtype, "pairs": pairs, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "partial": partial, "layout": layout, "mix": mix}


def _pages(name, rows_in, rows_out, page, cols, pool, mix=1):
    return {"name": name, "op": "pages", "rows_in": rows_in, "rows_out": rows_out, "page": page, "cols": cols,
            "pool": pool, "mix": mix}


def listed():
    # 32 heads of 128 (hidden size 4096), trees of 7 to 64 nodes, pages of 16 to 32 tokens.
    return [
        # the first answer tokens of a small model with a few drafted ones: latency only
        _attend("tree_first_tokens", "f32", 1, 7, 8, 8, 64, 16, 44),
        # a server's batch: lengths of 0 to 8192 mixed, trees of up to 32 nodes
        _attend("tree_mixed_batch", "bf16", 32, 32, 32, 8, 128, 16, 8192, lens="mixed", ragged=True),
        # one long document with a large tree: as many products as bytes
        _attend("tree_long", "f16", 1, 64, 32, 8, 128, 32, 100067),
        # a sliding window over wide heads, pages stored head by head that end inside a tile
        _attend("tree_window", "bf16", 8, 26, 16, 4, 256, 24, 10000, lens="mixed", window=1024, layout="head",
                ragged=True, mix=3),
        # one conversation's tree
        _plan("plan_one", 1, 26, 16, 4096),
        # a server's batch of the largest trees
        _plan("plan_batch", 128, 256, 16, 8192, mix=2),
        # one conversation, four drafted tokens accepted
        _compact("keep_one", "bf16", 1, 26, 4, 8, 128, 16),
        # a server's batch, up to eight accepted, pages stored head by head
        _compact("keep_batch", "f16", 192, 64, 8, 8, 128, 32, layout="head", mix=2),
        # one fork's last page, partly filled
        _copy("copy_one", "bf16", 1, 8, 128, 16, partial=True),
        # pages moved together before a pool shrinks
        _copy("copy_many", "bf16", 2047, 8, 128, 16, mix=2),
        # a server's step: some sequences end, some begin, some fork, the others grow or are cut back
        _pages("pages_step", 64, 64, 16, 512, 16384),
        # beams: every sequence forks from one of a few
        _pages("pages_beams", 256, 512, 16, 1024, 262144, mix=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "plan", "compact", "copy", "pages"])
    mix, dtype = rng.randrange(1 << 20), rng.choice(["f32", "bf16", "bf16", "f16"])
    page, layout = rng.choice([1, 8, 16, 16, 24, 32, 64, 128]), rng.choice(["token", "head"])
    if op == "attend":
        kv, head_dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
        group = rng.choice([1, 2, 4, 5, 7, 8, 8])
        nodes, batch = _log(rng, 1, 256), _log(rng, 1, 64)
        # the largest listed case's cache and products; 32-bit products are left to smaller trees
        room = 100067 * 8 * 128 * 2 // (kv * head_dim * WIDTH[dtype])
        room = min(room, 64 * 100067 * 32 * 128 // (nodes * kv * group * max(head_dim, 128)))
        if dtype == "f32":
            room = min(room, 64 * 6000 * 32 * 128 // (nodes * kv * group * head_dim))
        most = max(nodes + 1, min(100067, room // batch))
        window = rng.choice([0, 0, 0, _log(rng, 256, 4096)])
        c = _attend("", dtype, batch, nodes, kv * group, kv, head_dim, page, _log(rng, nodes + 1, most),
                    rng.choice(["full", "mixed", "mixed"]), window, layout, rng.random() < 0.5, mix)
    elif op == "plan":
        c = _plan("", _log(rng, 1, 128), _log(rng, 1, 256), page, _log(rng, 512, 8192),
                  rng.choice(["tree", "tree", "chain", "bush"]), mix)
    elif op == "compact":
        nodes = _log(rng, 2, 256)
        c = _compact("", dtype, _log(rng, 1, 192), nodes, _log(rng, 1, min(16, nodes)), rng.choice([1, 2, 4, 8]),
                     rng.choice([64, 80, 128, 128]), page, layout, mix)
    elif op == "copy":
        kv, head_dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128, 128, 256])
        room = 2047 * 16 * 8 * 128 * 2 // (page * kv * head_dim * WIDTH[dtype])
        c = _copy("", dtype, _log(rng, 1, max(1, min(2047, room))), kv, head_dim, page, rng.random() < 0.5, layout,
                  mix)
    else:
        rows = _log(rng, 1, 256)
        c = _pages("", rows, max(1, min(512, int(rows * rng.uniform(0.5, 2)))), max(8, page),
                   _log(rng, 16, 1024), _log(rng, 2048, 262144), mix)
    del c["name"]
    return c


def _lengths(case):
    """The sequences' committed tokens, from the case alone: with the tree they are max_len at most."""
    n, batch = case["max_len"] - case["nodes"], case["batch"]
    if case["lens"] == "full":
        return [n] * batch
    r = random.Random(case["mix"])
    got = [_log(r, 1, n) for _ in range(batch)]
    got[r.randrange(batch)] = n
    if batch >= 8:
        got[r.randrange(batch)] = 0  # nothing but the tree
    return got


def _counts(case):
    """How many nodes each sequence's tree has."""
    r = random.Random(case["mix"] + 1)
    if not case["ragged"]:
        return [case["nodes"]] * case["batch"]
    got = [r.randint(1, case["nodes"]) for _ in range(case["batch"])]
    if case["batch"] >= 8:
        got[r.randrange(case["batch"])] = 0  # a padded sequence
    return got


def _starts(case):
    """The first committed token that a root attends to."""
    w = case["window"]
    return [max(0, n + 1 - w) if w else 0 for n in _lengths(case)]


def work(case):
    if case["op"] == "attend":
        e, d, hq, hk = WIDTH[case["dtype"]], case["head_dim"], case["q_heads"], case["kv_heads"]
        b = f = 0
        for n, s, c in zip(_lengths(case), _starts(case), _counts(case)):
            if c:
                seen = n - s + c
                b += e * d * (2 * hk * seen + 2 * hq * c) + 4 * hq * c + 8 * c + 4 * -(-seen // case["page"]) + 8
                f += 4 * d * hq * c * (n - s + c / 2)
        return {"bytes": b, "flops": f}
    if case["op"] == "plan":
        b, n = case["batch"], case["nodes"]
        return {"bytes": b * n * (4 + 8 * -(-n // 64) + 8 + 8) + 8 * b, "flops": 0}
    if case["op"] == "compact":
        row = 2 * case["kv_heads"] * case["head_dim"] * WIDTH[case["dtype"]]
        moved = sum(j != i for p in _paths(case) for i, j in enumerate(p))
        return {"bytes": 2 * row * moved + 4 * moved + 8 * case["batch"], "flops": 0}
    if case["op"] == "copy":
        row = 2 * case["kv_heads"] * case["head_dim"] * WIDTH[case["dtype"]]
        return {"bytes": 2 * row * sum(_filled(case)) + 12 * case["pairs"], "flops": 0}
    rows = _moves(case)
    held = sum(-(-n // case["page"]) for n in rows["lens"])
    return {"bytes": 4 * (2 * case["pool"] + held + case["cols"] * case["rows_out"] + 7 * case["rows_out"]
                          + case["rows_in"]), "flops": 0}


# ------------------------------------------------------------------ inputs

def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _pool(gen, pages, case):
    """A cache's keys and values, both [pages, page, kv_heads, head_dim] to the user, stored token by token or head by head."""
    p, h, d, dtype = case["page"], case["kv_heads"], case["head_dim"], TYPES[case["dtype"]]
    if case["layout"] == "head":
        return [_randn(gen, (pages, h, p, d), dtype).transpose(1, 2) for _ in range(2)]
    return [_randn(gen, (pages, p, h, d), dtype) for _ in range(2)]


def _parents(r, nodes, shape):
    """A tree's parents, each before its children: a chain, a bush under the root, or in between."""
    if shape == "chain":
        return [i - 1 for i in range(nodes)]
    if shape == "bush":
        return [-1 if i < 4 else r.randrange(min(4, i)) for i in range(nodes)]
    return [-1] + [r.randrange(i // 4, i) for i in range(1, nodes)]


def _words(parents, nodes):
    """Each node's ancestors and itself, as words of 64 bits."""
    got, seen = [], []
    for i, p in enumerate(parents):
        seen.append((1 << i) | (seen[p] if p >= 0 else 0))
    for i in range(nodes):
        bits = seen[i] if i < len(seen) else 0
        for w in range(-(-nodes // 64)):
            x = (bits >> (64 * w)) & ((1 << 64) - 1)
            got.append(x - (1 << 64) if x >> 63 else x)
    return got


def _prepare_attend(case, gen, seed):
    page, batch, nodes = case["page"], case["batch"], case["nodes"]
    lens, counts, width = _lengths(case), _counts(case), -(-case["max_len"] // page)
    n, c = torch.tensor(lens, device=DEV), torch.tensor(counts, device=DEV)
    start = torch.tensor(_starts(case), device=DEV)
    r = random.Random(seed)
    words = [_words(_parents(r, k, "tree"), nodes) for k in counts]
    mask = torch.tensor(words, dtype=torch.int64).view(batch, nodes, -1).to(DEV)
    # pages held: those with a token that is attended to; the others' entries are -1
    col = torch.arange(width, device=DEV)
    held = (col * page < (n + c)[:, None]) & ((col + 1) * page > start[:, None])
    count = int(held.sum())
    pages = count + 3
    order = torch.randperm(pages, generator=gen, device=DEV)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    table[held] = order[:count].to(torch.int32)
    k, v = _pool(gen, pages, case)
    # what no token was written to holds anything, NaN among it
    stale = torch.ones((pages, page), dtype=torch.bool, device=DEV)
    at = (col[:, None] * page + torch.arange(page, device=DEV)) < (n + c)[:, None, None]
    stale[table[held].long()] = ~at[held]
    k[stale], v[stale] = math.nan, math.nan
    q = _randn(gen, (batch, nodes, case["q_heads"], case["head_dim"]), TYPES[case["dtype"]], 1.5)
    s = {"case": case, "q": q, "k": k, "v": v, "table": table, "lens": n.to(torch.int32),
         "counts": c.to(torch.int32), "mask": mask, "scale": case["head_dim"] ** -0.5, "out": torch.zeros_like(q),
         "lse": torch.zeros(q.shape[:3], dtype=torch.float32, device=DEV)}
    if own:
        import deterministic_fixed_order_gb300 as df
        s["cache"] = df.PagedCache(k, v)
        need = df.detfold_attn_tree_workspace_bytes(s["cache"], batch, nodes, case["q_heads"], case["max_len"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


def _prepare_plan(case, gen, seed):
    page, batch, nodes = case["page"], case["batch"], case["nodes"]
    r = random.Random(seed)
    width = -(-(case["max_len"] + nodes) // page)
    lens = [r.randrange(case["max_len"]) for _ in range(batch)]
    counts = [r.randint(max(1, nodes // 2), nodes) for _ in range(batch)]
    parents = [p + [-1] * (nodes - len(p)) for p in (_parents(r, c, case["shape"]) for c in counts)]
    table = torch.randperm(batch * width, generator=gen, device=DEV).view(batch, width).to(torch.int32)
    i32 = {"dtype": torch.int32, "device": DEV}
    i64 = {"dtype": torch.int64, "device": DEV}
    return {"case": case, "parents": torch.tensor(parents, **i32), "counts": torch.tensor(counts, **i32),
            "lens": torch.tensor(lens, **i32), "table": table,
            "mask": torch.empty(batch, nodes, -(-nodes // 64), **i64), "positions": torch.empty(batch, nodes, **i64),
            "slots": torch.empty(batch, nodes, **i64)}


def _paths(case):
    """The accepted nodes of each sequence's tree, from the root down: their numbers ascend."""
    r = random.Random(case["mix"])
    got = []
    for _ in range(case["batch"]):
        length = r.randint(1, case["path"]) if case["batch"] > 1 else case["path"]
        got.append([0] + sorted(r.sample(range(1, case["nodes"]), length - 1)))
    return got


def _prepare_compact(case, gen, seed):
    page, batch, nodes = case["page"], case["batch"], case["nodes"]
    r = random.Random(seed)
    room = 4 * page + nodes
    width = -(-room // page)
    lens = [r.randrange(4 * page) for _ in range(batch)]
    pages = batch * width + 3
    table = torch.randperm(pages, generator=gen, device=DEV)[:batch * width].view(batch, width).to(torch.int32)
    k, v = _pool(gen, pages, case)
    paths = _paths(case)
    path = torch.tensor([p + [-1] * (case["path"] - len(p)) for p in paths], dtype=torch.int32, device=DEV)
    s = {"case": case, "k": k, "v": v, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "path": path, "path_lens": torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)}
    if own:
        import deterministic_fixed_order_gb300 as df
        s["cache"] = df.PagedCache(k, v)
    return s


def _filled(case):
    """How many rows of each page are copied."""
    r = random.Random(case["mix"])
    return [r.randint(1, case["page"]) if case["partial"] else case["page"] for _ in range(case["pairs"])]


def _prepare_copy(case, gen, seed):
    pairs = case["pairs"]
    order = torch.randperm(2 * pairs + 3, generator=gen, device=DEV).to(torch.int32)
    k, v = _pool(gen, 2 * pairs + 3, case)
    s = {"case": case, "k": k, "v": v, "src": order[:pairs].contiguous(), "dst": order[pairs:2 * pairs].contiguous(),
         "rows": torch.tensor(_filled(case), dtype=torch.int32, device=DEV) if case["partial"] else None}
    if own:
        import deterministic_fixed_order_gb300 as df
        s["cache"] = df.PagedCache(k, v)
    return s


def _moves(case):
    """What a step does to each sequence: the row that it goes on from, the tokens that it keeps, and those that it needs room for."""
    r = random.Random(case["mix"])
    page, n, m = case["page"], case["rows_in"], case["rows_out"]
    # the pool holds every sequence twice over, or the sequences are shorter
    most = max(1, min(case["cols"], case["pool"] // (2 * max(n, m)) - 1)) * page
    lens = [_log(r, 1, most) for _ in range(n)]
    origin, keep, want = [], [], []
    for b in range(m):
        what = r.random()
        f = b if b < n and what < 0.7 else r.randrange(n)
        if what < 0.55 or b >= n:
            k = lens[f]                      # goes on, or forks
        elif what < 0.7:
            k = r.randint(0, lens[f])        # is cut back to what was accepted
        elif what < 0.8:
            f, k = -1, 0                     # begins
        else:
            k = lens[f]
        w = 0 if what > 0.95 else min(most, _log(r, 1, most) if f < 0 else k + r.randint(0, 64))
        if w == 0:
            f, k = -1, 0                     # ended: an empty row
        origin.append(f)
        keep.append(min(k, w))
        want.append(w)
    return {"lens": lens, "origin": origin, "keep": keep, "want": want}


def _prepare_pages(case, gen, seed):
    page, n, cols, pool = case["page"], case["rows_in"], case["cols"], case["pool"]
    rows = _moves(case)
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    lens = torch.tensor(rows["lens"], dtype=torch.int32, device=DEV)
    held = (lens.long() + page - 1) // page
    col = torch.arange(cols, device=DEV)
    first = torch.cumsum(held, 0) - held
    mine = col < held[:, None]
    table = torch.where(mine, order[torch.where(mine, first[:, None] + col, 0)], -1)
    # every eighth sequence shares its full pages with the one before it (a common prompt)
    shared = (torch.arange(n, device=DEV) % 8 == 7)[:, None] & mine & (((col + 1) * page) <= lens[:, None])
    shared[1:] &= (((col + 1) * page) <= lens[:-1, None])
    shared[:1] = False
    table = torch.where(shared, table.roll(1, 0), table).contiguous()
    refs = torch.zeros(pool, dtype=torch.int32, device=DEV)
    refs.index_add_(0, table[mine].long(), torch.ones(int(mine.sum()), dtype=torch.int32, device=DEV))
    # pages that something else holds (kept prompts), some of them sequences' too
    kept = torch.randint(0, pool, (pool // 16,), generator=gen, device=DEV)
    refs.index_add_(0, kept, torch.ones_like(kept, dtype=torch.int32))
    i32 = {"dtype": torch.int32, "device": DEV}
    m = case["rows_out"]
    return {"case": case, "refs": refs, "table": table, "lens": lens,
            "origin": torch.tensor(rows["origin"], **i32), "keep": torch.tensor(rows["keep"], **i32),
            "want": torch.tensor(rows["want"], **i32), "refs_out": torch.empty_like(refs),
            "table_out": torch.empty(m, cols, **i32), "lens_out": torch.empty(m, **i32),
            "copy_src": torch.empty(m, **i32), "copy_dst": torch.empty(m, **i32), "copy_rows": torch.empty(m, **i32)}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    made = {"attend": _prepare_attend, "plan": _prepare_plan, "compact": _prepare_compact, "copy": _prepare_copy,
            "pages": _prepare_pages}
    return made[case["op"]](case, gen, seed)


# ------------------------------------------------------------------ plain forms

def _bits(mask, count):
    """Words of 64 bits as truth values."""
    bit = torch.arange(64, device=DEV)
    return ((mask[..., None] >> bit) & 1).flatten(-2)[..., :count].bool()


def _seen(s):
    """[batch, nodes, max_len]: which tokens of its sequence a node attends to."""
    case, n, c = s["case"], s["lens"].long(), s["counts"].long()
    nodes, pos = case["nodes"], torch.arange(case["max_len"], device=DEV)
    tree = _bits(s["mask"], nodes) & (torch.arange(nodes, device=DEV) < c[:, None])[:, None]
    far = (pos - n[:, None])[:, None].expand(-1, nodes, -1)
    drafted = (far >= 0) & (far < nodes) & tree.gather(2, far.clamp(0, nodes - 1))
    before = far < 0
    if case["window"]:
        before = before & (far >= tree.sum(2).clamp_min(1)[..., None] - case["window"])
    return drafted | before


def _plain_attend(s):
    case, q, hk, page = s["case"], s["q"], s["case"]["kv_heads"], s["case"]["page"]
    seen = _seen(s)
    live = torch.arange(case["nodes"], device=DEV) < s["counts"][:, None]
    seen &= live[..., None]
    pos = torch.arange(case["max_len"], device=DEV)
    any_seen = seen.any(1)
    at = torch.where(any_seen, s["table"].long()[:, pos // page], 0)
    here = any_seen[:, :, None, None]
    k = torch.where(here, s["k"][at, pos % page], 0).float()
    v = torch.where(here, s["v"][at, pos % page], 0).float()
    b, t, hq, d = q.shape
    g = hq // hk
    qg = q.float().view(b, t, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, t * g, d)
    scores = torch.matmul(qg, k.permute(0, 2, 3, 1)).view(b, hk, t, g, -1) * s["scale"]
    scores = torch.where(seen[:, None, :, None], scores, NEG)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == NEG, 0, top)
    p = torch.exp(scores.sub_(top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, t * g, -1), v.permute(0, 2, 1, 3)).view(b, hk, t, g, d)
    o = (o / torch.where(total == 0, 1, total)).permute(0, 2, 1, 3, 4).reshape(q.shape)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(b, t, hq)
    # rows behind a sequence's last node stay as they were
    return {"out": torch.where(live[..., None, None], o.to(q.dtype), s["out"]),
            "lse": torch.where(live[..., None], lse, s["lse"])}


def _plain_plan(s):
    case, parents, n = s["case"], s["parents"].long(), s["lens"].long()
    nodes, page = case["nodes"], case["page"]
    i = torch.arange(nodes, device=DEV)
    live = i < s["counts"][:, None]
    reach = (i[:, None] == i) | ((i == parents[..., None]) & live[..., None])
    for _ in range((nodes - 1).bit_length()):  # paths of twice the length each time
        reach = torch.matmul(reach.float(), reach.float()) > 0
    reach &= live[..., None]
    words = -(-nodes // 64)
    padded = torch.zeros(reach.shape[:2] + (64 * words,), dtype=torch.int64, device=DEV)
    padded[..., :nodes] = reach
    mask = (padded.view(reach.shape[:2] + (words, 64)) << torch.arange(64, device=DEV)).sum(-1)
    at = n[:, None] + i
    slots = s["table"].long().gather(1, at // page) * page + at % page
    return {"mask": mask, "positions": torch.where(live, n[:, None] + reach.sum(-1) - 1, 0),
            "slots": torch.where(live, slots, -1)}


def _plain_compact(s):
    page, n, path = s["case"]["page"], s["lens"].long(), s["path"].long()
    i = torch.arange(path.shape[1], device=DEV)
    live = i < s["path_lens"][:, None]
    table = s["table"].long()
    src, dst = (n[:, None] + path)[live], (n[:, None] + i)[live]
    row = torch.arange(len(n), device=DEV)[:, None].expand_as(path)[live]
    a, b = (table[row, src // page], src % page), (table[row, dst // page], dst % page)
    s["k"][b], s["v"][b] = s["k"][a], s["v"][a]
    return {"k": s["k"], "v": s["v"]}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    if s["rows"] is None:
        s["k"][dst], s["v"][dst] = s["k"][src], s["v"][src]
    else:
        take = (torch.arange(s["case"]["page"], device=DEV) < s["rows"][:, None])[:, :, None, None]
        s["k"][dst] = torch.where(take, s["k"][src], s["k"][dst])
        s["v"][dst] = torch.where(take, s["v"][src], s["v"][dst])
    return {"k": s["k"], "v": s["v"]}


def _plain_pages(s):
    case, page, table = s["case"], s["case"]["page"], s["table"].long()
    origin, keep, want, lens = (s[x].long() for x in ("origin", "keep", "want", "lens"))
    col = torch.arange(case["cols"], device=DEV)
    up = lambda x: (x + page - 1) // page  # noqa: E731
    old = col < up(lens)[:, None]
    kept = col < up(keep)[:, None]
    from_row = table[origin.clamp_min(0)]
    one = torch.ones(1, dtype=torch.int64, device=DEV)
    cnt = s["refs"].long()
    cnt.index_add_(0, table[old], -one.expand(int(old.sum())))
    cnt.index_add_(0, from_row[kept], one.expand(int(kept.sum())))
    # a page that a row goes on writing into is its own, or is copied
    last = up(keep) - 1
    partial = (keep % page != 0) & (want > keep)
    held = from_row.gather(1, last.clamp_min(0)[:, None])[:, 0]
    copies = partial & (cnt[held.clamp_min(0)] > 1)
    need = up(want) - up(keep) + copies
    ends = torch.cumsum(need, 0)
    free = torch.nonzero(cnt == 0)[:, 0]
    served = (need == 0) | (ends <= len(free))
    copies &= served
    fresh = (col >= (up(keep) - copies.long())[:, None]) & (col < up(want)[:, None]) & served[:, None]
    nth = (ends - need)[:, None] + col - (up(keep) - copies.long())[:, None]
    new = torch.where(fresh, free[torch.where(fresh, nth, 0)] if len(free) else 0, torch.where(kept, from_row, -1))
    cnt.index_add_(0, held[copies], -one.expand(int(copies.sum())))
    cnt.index_add_(0, new[fresh], one.expand(int(fresh.sum())))
    src = torch.where(copies, held, -1)
    dst = torch.where(copies, new.gather(1, last.clamp_min(0)[:, None])[:, 0], -1)
    got = {"refs": cnt, "table": new, "lens": torch.where(served, want, keep), "copy_src": src, "copy_dst": dst,
           "copy_rows": torch.where(copies, keep % page, 0)}
    return {x: y.to(torch.int32) for x, y in got.items()}


# ------------------------------------------------------------------ the package's operators

def _own_attend(s):
    import deterministic_fixed_order_gb300 as df
    case = s["case"]
    df.detfold_attn_tree(s["out"], s["q"], s["cache"], s["table"], s["lens"], s["mask"], case["max_len"], s["scale"],
                         node_counts=s["counts"], window=case["window"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_plan(s):
    import deterministic_fixed_order_gb300 as df
    case = s["case"]
    df.detfold_tree_plan(s["mask"], s["parents"], s["lens"], s["table"], case["page"], case["batch"] * s["table"].shape[1],
                         node_counts=s["counts"], positions=s["positions"], slots=s["slots"])
    return {"mask": s["mask"], "positions": s["positions"], "slots": s["slots"]}


def _own_compact(s):
    import deterministic_fixed_order_gb300 as df
    df.detfold_kv_compact(s["cache"], s["table"], s["lens"], s["path"], s["path_lens"])
    return {"k": s["k"], "v": s["v"]}


def _own_copy(s):
    import deterministic_fixed_order_gb300 as df
    df.detfold_kv_copy_pages(s["cache"], s["src"], s["dst"], rows=s["rows"])
    return {"k": s["k"], "v": s["v"]}


def _own_pages(s):
    import deterministic_fixed_order_gb300 as df
    df.detfold_pages_step(s["refs_out"], s["table_out"], s["lens_out"], s["copy_src"], s["copy_dst"], s["copy_rows"],
                          s["refs"], s["table"], s["lens"], s["origin"], s["keep"], s["want"], s["case"]["page"])
    return {"refs": s["refs_out"], "table": s["table_out"], "lens": s["lens_out"], "copy_src": s["copy_src"],
            "copy_dst": s["copy_dst"], "copy_rows": s["copy_rows"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "plan": _own_plan, "compact": _own_compact, "copy": _own_copy,
                "pages": _own_pages}[op](state)
    return {"attend": _plain_attend, "plan": _plain_plan, "compact": _plain_compact, "copy": _plain_copy,
            "pages": _plain_pages}[op](state)


# ------------------------------------------------------------------ 64 bits

def _exact_attend(s):
    case = s["case"]
    out, lse = s["out"].double(), s["lse"].double()
    hk, page, w = case["kv_heads"], case["page"], case["window"]
    g, nodes = case["q_heads"] // hk, case["nodes"]
    for b, (n, start, c) in enumerate(zip(_lengths(case), _starts(case), _counts(case))):
        if not c:
            continue
        t = torch.arange(start, n + c, device=DEV)
        at = s["table"][b, t // page].long(), t % page
        anc = torch.zeros(c, nodes, dtype=torch.bool, device=DEV)
        for i in range(nodes):
            anc[:, i] = (s["mask"][b, :c, i // 64] >> (i % 64)) % 2 != 0
        depth = anc.sum(1) - 1
        hidden = torch.cat([(t[:n - start] <= n + depth[:, None] - w) if w else
                            torch.zeros(c, n - start, dtype=torch.bool, device=DEV), ~anc[:, :c]], 1)
        for h in range(hk):
            k, v = s["k"][at][:, h].double(), s["v"][at][:, h].double()
            for j in range(h * g, (h + 1) * g):
                x = (s["q"][b, :c, j].double() @ k.T * s["scale"]).masked_fill(hidden, NEG)
                lse[b, :c, j] = torch.logsumexp(x, 1)
                out[b, :c, j] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}


def _exact_moved(s, moves):
    """The cache in 64 bits after rows went from (page, row) to (page, row), all read before any is written."""
    k, v = s["k"].double(), s["v"].double()
    new = [(to, k[at].clone(), v[at].clone()) for at, to in moves]
    for to, x, y in new:
        k[to], v[to] = x, y
    return {"k": k, "v": v}


def _exact_compact(s):
    page, moves = s["case"]["page"], []
    for n, row, path in zip(s["lens"].tolist(), s["table"].tolist(), _paths(s["case"])):
        for i, j in enumerate(path):
            moves.append(((row[(n + j) // page], (n + j) % page), (row[(n + i) // page], (n + i) % page)))
    return _exact_moved(s, moves)


def _exact_copy(s):
    pairs = zip(s["src"].tolist(), s["dst"].tolist(), _filled(s["case"]))
    return _exact_moved(s, [((a, slice(0, n)), (b, slice(0, n))) for a, b, n in pairs])


def exact(case, seed):
    made = {"attend": _exact_attend, "compact": _exact_compact, "copy": _exact_copy}
    return made[case["op"]](prepare(case, seed)) if case["op"] in made else None
