"""Measured cases of the decode-step operators: appending keys and values to a
paged cache with the position rotation applied on the way, attention of one new
token over that cache, and the join of W ranks' partial attentions.

Each operator is given twice: in plain form (elementary torch operations in
32 bits, rounded once at the end) and, where ``own`` is true, as the calls that a
user makes of this package. ``exact`` computes the same from the definitions
in 64 bits.
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

def _decode(name, dtype, batch, q_heads, kv_heads, head_dim, page, max_len, lens="full", window=0,
            layout="token", mix=1):
    return {"name": name, "op": "decode", "dtype": dtype, "batch": batch, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "max_len": max_len,
            "lens": lens, "window": window, "layout": layout, "mix": mix}


def _append(name, dtype, tokens, q_heads, kv_heads, head_dim, rot, style, page, padding=False,
            layout="token", mix=1):
    return {"name": name, "op": "append", "dtype": dtype, "tokens": tokens, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "rot": rot, "style": style, "page": page,
            "padding": padding, "layout": layout, "mix": mix}


def _join(name, dtype, world, rows, heads, head_dim, mix=1):
    return {"name": name, "op": "join", "dtype": dtype, "world": world, "rows": rows, "heads": heads,
            "head_dim": head_dim, "mix": mix}


def listed():
    # Hidden size 4096 (the decode join's payload) as 32 heads of 128; world sizes 2 to 8.
    return [
        # the first answer tokens of a small model: latency only
        _decode("decode_first_tokens", "f32", 1, 8, 8, 64, 16, 37),
        # one conversation, few pages: split over the length or idle
        _decode("decode_one_chat", "bf16", 1, 32, 8, 128, 16, 4093),
        # a server's batch: lengths of 0 to 8192 mixed, odd ones among them
        _decode("decode_mixed_batch", "bf16", 64, 32, 8, 128, 16, 8192, lens="mixed"),
        # one long document: the length alone fills the card
        _decode("decode_long", "f16", 1, 32, 8, 128, 64, 131071),
        # a rank of an 8-way split: one shared key-value head, pages stored head by head
        _decode("decode_rank_shard", "bf16", 32, 8, 1, 128, 32, 4096, lens="mixed", layout="head", mix=2),
        # a sliding window over wide heads, pages that end inside a tile
        _decode("decode_window", "f16", 24, 16, 4, 256, 24, 10000, lens="mixed", window=1024, mix=3),
        # 32-bit cache, a head of keys for every head of queries, odd head size
        _decode("decode_f32", "f32", 16, 12, 12, 80, 16, 2047, lens="mixed", mix=4),
        # one token of one conversation: latency only
        _append("append_one", "bf16", 1, 32, 8, 128, 128, "half", 16),
        # one token each of a server's batch, padded for a captured graph; part of the head rotated
        _append("append_batch", "f16", 192, 16, 4, 256, 64, "pairs", 32, padding=True, layout="head"),
        # a prompt
        _append("append_prompt", "bf16", 16381, 32, 8, 128, 128, "half", 16),
        # two ranks' halves of one decode step
        _join("join_step", "f32", 2, 1, 32, 128),
        # eight ranks' parts of a prompt's rows
        _join("join_rows", "bf16", 8, 4099, 32, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    op = rng.choice(["decode", "decode", "decode", "append", "append", "join"])
    mix = rng.randrange(1 << 20)
    if op == "decode":
        kv, head_dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
        group = rng.choice([1, 2, 4, 5, 7, 8, 8, 16])
        room = 131071 * 8 * 128 * 2 // (kv * head_dim * WIDTH[dtype])  # tokens of the largest listed case
        batch = _log(rng, 1, 128)
        max_len = _log(rng, 1, min(131071, room // batch))
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        c = _decode("", dtype, batch, kv * group, kv, head_dim, rng.choice([1, 8, 16, 16, 24, 32, 64, 256]),
                    max_len, rng.choice(["full", "mixed", "mixed"]), window, rng.choice(["token", "head"]), mix)
    elif op == "append":
        kv, head_dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128, 128, 256])
        group = rng.choice([1, 2, 4, 8])
        room = 16381 * 48 * 128 * 2 // ((group + 2) * kv * head_dim * WIDTH[dtype])
        tokens = _log(rng, 1, min(16381, room))
        rot = rng.choice([head_dim, head_dim, head_dim // 2, 2 * (head_dim // 8)])
        c = _append("", dtype, tokens, kv * group, kv, head_dim, rot, rng.choice(["half", "half", "pairs"]),
                    rng.choice([1, 8, 16, 24, 32, 64]), rng.random() < 0.5, rng.choice(["token", "head"]), mix)
    else:
        world, heads, head_dim = rng.choice([2, 3, 4, 6, 8]), rng.choice([1, 5, 8, 32]), rng.choice([40, 64, 128, 128, 256])
        room = 8 * 4099 * 32 * 128 * 2 // (world * heads * head_dim * WIDTH[dtype])
        c = _join("", dtype, world, _log(rng, 1, min(32768, room)), heads, head_dim, mix)
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths, from the case alone."""
    n, batch = case["max_len"], case["batch"]
    if case["lens"] == "full":
        return [n] * batch
    r = random.Random(case["mix"])
    got = [_log(r, 1, n) for _ in range(batch)]
    got[r.randrange(batch)] = n
    if batch >= 8:
        got[r.randrange(batch)] = 0  # a padded row
    return got


def _seen(case):
    """How many cached tokens each sequence's new token attends to."""
    w = case["window"]
    return [min(n, w) if w else n for n in _lengths(case)]


def work(case):
    e = WIDTH[case["dtype"]]
    d = case["head_dim"]
    if case["op"] == "decode":
        seen, hq, hk, b = sum(_seen(case)), case["q_heads"], case["kv_heads"], case["batch"]
        pages = sum(-(-n // case["page"]) for n in _seen(case))
        return {"bytes": e * d * (2 * hk * seen + 2 * hq * b) + 4 * b * hq + 4 * pages + 4 * b,
                "flops": 4 * hq * d * seen}
    if case["op"] == "append":
        t, hq, hk, r = case["tokens"], case["q_heads"], case["kv_heads"], case["rot"]
        return {"bytes": e * t * d * (2 * hq + 4 * hk) + 4 * t * r + 16 * t, "flops": 3 * t * r * (hq + hk)}
    rows, w = case["rows"] * case["heads"], case["world"]
    return {"bytes": (e * d + 4) * rows * (w + 1), "flops": 2 * rows * w * (d + 4)}


# ------------------------------------------------------------------ inputs

def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _pool(gen, pages, case, dtype):
    """A cache's keys and values, both [pages, page, kv_heads, head_dim] to the user, stored token by token or head by head."""
    p, h, d = case["page"], case["kv_heads"], case["head_dim"]
    if case["layout"] == "head":
        return [_randn(gen, (pages, h, p, d), dtype).transpose(1, 2) for _ in range(2)]
    return [_randn(gen, (pages, p, h, d), dtype) for _ in range(2)]


def _prepare_decode(case, gen):
    dtype, page, batch = TYPES[case["dtype"]], case["page"], case["batch"]
    lens, width = _lengths(case), max(1, -(-case["max_len"] // page))
    n = torch.tensor(lens, device=DEV)
    start = n - torch.tensor(_seen(case), device=DEV)
    # pages still held: those with a token that is attended to; the others' entries are -1
    col = torch.arange(width, device=DEV)
    held = (col * page < n[:, None]) & ((col + 1) * page > start[:, None])
    count = int(held.sum())
    pages = count + 3
    order = torch.randperm(pages, generator=gen, device=DEV)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    table[held] = order[:count].to(torch.int32)
    k, v = _pool(gen, pages, case, dtype)
    # what no token was written to holds anything, NaN among it
    stale = torch.ones((pages, page), dtype=torch.bool, device=DEV)
    at = (col[:, None] * page + torch.arange(page, device=DEV)) < n[:, None, None]
    stale[table[held].long()] = ~at[held]
    k[stale], v[stale] = math.nan, math.nan
    q = _randn(gen, (batch, case["q_heads"], case["head_dim"]), dtype, 1.5)
    s = {"case": case, "q": q, "k": k, "v": v, "table": table, "lens": n.to(torch.int32),
         "scale": case["head_dim"] ** -0.5}
    if own:
        import deterministic_fixed_order_gb300 as df
        s["cache"] = df.PagedCache(k, v)
        s["out"] = torch.empty_like(q)
        s["lse"] = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
        need = df.detfold_attn_decode_workspace_bytes(s["cache"], batch, case["q_heads"], case["max_len"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


def _prepare_append(case, gen):
    dtype, page, t = TYPES[case["dtype"]], case["page"], case["tokens"]
    hq, hk, d, r = case["q_heads"], case["kv_heads"], case["head_dim"], case["rot"]
    pages = -(-t // page) + max(4, -(-64 // page))
    k, v = _pool(gen, pages, case, dtype)
    # one projection's output: a token's queries, keys and values lie side by side
    qkv = _randn(gen, (t, hq + 2 * hk, d), dtype)
    limit = t + 4096
    freq = torch.pow(10000.0, -torch.arange(r // 2, device=DEV, dtype=torch.float64) * 2 / r)
    angle = torch.arange(limit, device=DEV, dtype=torch.float64)[:, None] * freq
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    first = int(torch.randint(0, 4096, (1,), generator=gen, device=DEV))
    if t > 512:  # a prompt: its positions in turn, its pages anywhere
        positions = first + torch.arange(t, device=DEV)
        order = torch.randperm(pages, generator=gen, device=DEV)
        i = torch.arange(t, device=DEV)
        slots = order[i // page] * page + i % page
    else:  # a token each of several sequences
        positions = torch.randint(0, limit, (t,), generator=gen, device=DEV)
        slots = torch.randperm(pages * page, generator=gen, device=DEV)[:t]
    if case["padding"]:
        positions[t - t // 8:], slots[t - t // 8:] = 0, -1
    s = {"case": case, "k": k, "v": v, "new_q": qkv[:, :hq], "new_k": qkv[:, hq:hq + hk],
         "new_v": qkv[:, hq + hk:], "cos_sin": cos_sin, "positions": positions, "slots": slots}
    if own:
        import deterministic_fixed_order_gb300 as df
        s["cache"] = df.PagedCache(k, v)
        s["rope"] = df.Rope(cos_sin, interleaved=case["style"] == "pairs")
        s["q_out"] = torch.empty((t, hq, d), dtype=dtype, device=DEV)
    return s


def _prepare_join(case, gen):
    w, dtype, shape = case["world"], TYPES[case["dtype"]], (case["rows"], case["heads"])
    parts = [_randn(gen, shape + (case["head_dim"],), dtype) for _ in range(w)]
    lses = [torch.randn(shape, generator=gen, device=DEV) * 2 + 6 for _ in range(w)]
    # a rank whose part of a row is empty; a row that is empty on every rank
    empty = torch.rand((w,) + shape, generator=gen, device=DEV) < 0.1
    empty |= torch.rand(shape, generator=gen, device=DEV) < 0.02
    empty[0, 0, 0] = False
    for r, (part, lse) in enumerate(zip(parts, lses)):
        lse[empty[r]] = NEG
        part[empty[r]] = math.nan
    s = {"case": case, "parts": parts, "lses": lses}
    if own:
        s["out"] = torch.empty_like(parts[0])
        s["lse"] = torch.empty_like(lses[0])
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"decode": _prepare_decode, "append": _prepare_append, "join": _prepare_join}[case["op"]](case, gen)


# ------------------------------------------------------------------ plain forms

def _plain_decode(s):
    case, q, n = s["case"], s["q"], s["lens"].long()
    page, w, hk = case["page"], case["window"], case["kv_heads"]
    pos = torch.arange(case["max_len"], device=DEV)
    seen = pos < n[:, None]
    if w:
        seen &= pos >= n[:, None] - w
    at = torch.where(seen, s["table"].long()[:, pos // page], 0)
    here = seen[:, :, None, None]
    k = torch.where(here, s["k"][at, pos % page], 0).float()
    v = torch.where(here, s["v"][at, pos % page], 0).float()
    qg = q.float().view(q.shape[0], hk, -1, q.shape[2])
    scores = torch.matmul(qg, k.permute(0, 2, 3, 1)) * s["scale"]
    scores = torch.where(seen[:, None, None, :], scores, NEG)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == NEG, 0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1, total)
    lse = (top + torch.log(total)).view(q.shape[:2])
    return {"out": o.view(q.shape).to(q.dtype), "lse": lse}


def _plain_rotate(x, cos, sin, r, style):
    x = x.float()
    if style == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_append(s):
    case, r = s["case"], s["case"]["rot"]
    row = s["cos_sin"][s["positions"]][:, None]
    cos, sin = row[..., :r // 2], row[..., r // 2:]
    q = _plain_rotate(s["new_q"], cos, sin, r, case["style"]).to(s["new_q"].dtype)
    k = _plain_rotate(s["new_k"], cos, sin, r, case["style"]).to(s["new_k"].dtype)
    v, slots = s["new_v"], s["slots"]
    if case["padding"]:
        live = slots >= 0
        k, v, slots = k[live], v[live], slots[live]
    at = (slots // case["page"], slots % case["page"])
    s["k"][at] = k
    s["v"][at] = v
    return {"q": q, "k": s["k"], "v": s["v"]}


def _plain_join(s):
    parts, lses = torch.stack(s["parts"]).float(), torch.stack(s["lses"])
    top = lses.amax(0)
    top = torch.where(top == NEG, 0, top)
    w = torch.exp(lses - top)
    total = w.sum(0)
    o = torch.where((w > 0)[..., None], parts, 0).mul_(w[..., None]).sum(0)
    o = o / torch.where(total == 0, 1, total)[..., None]
    return {"out": o.to(s["parts"][0].dtype), "lse": top + torch.log(total)}


# ------------------------------------------------------------------ the package's operators

def _own_decode(s):
    import deterministic_fixed_order_gb300 as df
    case = s["case"]
    df.detfold_attn_decode(s["out"], s["q"], s["cache"], s["table"], s["lens"], case["max_len"], s["scale"],
                           window=case["window"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    import deterministic_fixed_order_gb300 as df
    df.detfold_kv_append(s["cache"], s["new_k"], s["new_v"], s["slots"], rope=s["rope"],
                         positions=s["positions"], q=s["new_q"], q_out=s["q_out"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _own_join(s):
    import deterministic_fixed_order_gb300 as df
    df.detfold_attn_join(s["out"], s["parts"], s["lses"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"decode": _own_decode, "append": _own_append, "join": _own_join}[op](state)
    return {"decode": _plain_decode, "append": _plain_append, "join": _plain_join}[op](state)


# ------------------------------------------------------------------ 64 bits

def _exact_decode(s):
    case, hk = s["case"], s["case"]["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], NEG, dtype=torch.float64, device=DEV)
    for b, (n, seen) in enumerate(zip(_lengths(case), _seen(case))):
        if not n:
            continue
        t = torch.arange(n - seen, n, device=DEV)
        slot = s["table"][b, t // case["page"]].long(), t % case["page"]
        k, v = s["k"][slot].double(), s["v"][slot].double()
        for h in range(hk):
            g = slice(h * case["q_heads"] // hk, (h + 1) * case["q_heads"] // hk)
            x = (k[:, h] @ s["q"][b, g].double().T) * s["scale"]  # [tokens, heads]
            lse[b, g] = torch.logsumexp(x, 0)
            out[b, g] = torch.softmax(x, 0).T @ v[:, h]
    return {"out": out, "lse": lse}


def _exact_append(s):
    case, r = s["case"], s["case"]["rot"]
    angle = s["cos_sin"].double()[s["positions"]]
    turn = torch.complex(angle[:, :r // 2], angle[:, r // 2:])[:, None]

    def rotate(x):
        y = x.double().clone()
        ia = torch.arange(r // 2, device=DEV) * (2 if case["style"] == "pairs" else 1)
        ib = ia + (1 if case["style"] == "pairs" else r // 2)
        z = torch.complex(y[..., ia], y[..., ib]) * turn
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    live = s["slots"] >= 0
    slots = s["slots"][live]
    at = (slots // case["page"], slots % case["page"])
    k, v = s["k"].double(), s["v"].double()
    k[at], v[at] = rotate(s["new_k"])[live], s["new_v"][live].double()
    return {"q": rotate(s["new_q"]), "k": k, "v": v}


def _exact_join(s):
    lses = [x.double() for x in s["lses"]]
    lse = torch.logsumexp(torch.stack(lses), 0)
    out = torch.zeros(s["parts"][0].shape, dtype=torch.float64, device=DEV)
    for part, x in zip(s["parts"], lses):
        share = torch.where(x == NEG, 0, torch.exp(x - lse))[..., None]
        out += torch.where(share > 0, part.double() * share, 0)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "append": _exact_append, "join": _exact_join}[case["op"]](s)
