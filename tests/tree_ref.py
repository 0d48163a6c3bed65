"""The operators of a step with drafted tokens from their definitions, on the CPU: the
attention in 64 bits with a bound on what a binary32 computation may be off by, the
others in whole numbers.

Bounds, as in attn_ref: u = 2^-24, 2u a step for matrix units, which may truncate. A score
is a dot product of D terms times scale, and its exponent is taken with two more
roundings of |s|: off by ds = (D + 4) 2u scale sum|q||k| + 4u |s|. A weight is off by a
factor 1 + ds + 8u, sums of n terms by n + 64 roundings of 2u, and 16-bit weights are held in
two parts (2^-16). With V = max |v| over what the row attends to, twice for the quotient's
two sides:
    |o - exact| <= 2 V (ds + 8u + (n + 64) 2u + 2^-16 [16-bit types]) + r |exact|
"""
from __future__ import annotations

import random

import torch

from attn_ref import U, final_round


def parents_of(seed, nodes, shape="tree"):
    r = random.Random(seed)
    if shape == "chain":
        return [i - 1 for i in range(nodes)]
    if shape == "roots":
        return [-1] * nodes
    return [-1] + [r.randrange(-1 if r.random() < 0.1 else i // 3, i) for i in range(1, nodes)]


def ancestors(parents):
    """Per node, the set of itself and its ancestors."""
    got = []
    for i, p in enumerate(parents):
        got.append({i} | (got[p] if p >= 0 else set()))
    return got


def words(sets, nodes):
    """Sets of nodes as [nodes, words] int64."""
    out = torch.zeros(nodes, -(-nodes // 64), dtype=torch.int64)
    for i, s in enumerate(sets):
        for w in range(out.shape[1]):
            x = sum(1 << (j - 64 * w) for j in s if 64 * w <= j < 64 * w + 64)
            out[i, w] = x - (1 << 64) if x >> 63 else x
    return out


def sees(mask_row, c):
    """[c] truth values of one node's words."""
    return torch.tensor([(int(mask_row[j // 64]) >> (j % 64)) & 1 == 1 for j in range(c)], dtype=torch.bool)


def attend(q, k, v, table, lens, mask, scale, counts=None, window=0):
    """(out, lse, out bound, lse bound, live); rows that are not live are left as they were."""
    batch, nodes, hq, width = q.shape
    page, hk = k.shape[1], k.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full((batch, nodes, hq), float("-inf"), dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    live = torch.zeros(batch, nodes, dtype=torch.bool)
    g = hq // hk
    for b in range(batch):
        n, c = int(lens[b]), nodes if counts is None else int(counts[b])
        live[b, :c] = True
        if c == 0:
            continue
        first = max(0, n + 1 - window) if window else 0
        t = torch.arange(first, n + c)
        pages = table[b].cpu().long()[t // page]
        at = (pages.to(k.device), (t % page).to(k.device))
        kk, vv, qq = k[at].double().cpu(), v[at].double().cpu(), q[b, :c].double().cpu()
        for i in range(c):
            tree = sees(mask[b, i].cpu(), c)
            p = n + max(1, int(tree.sum())) - 1
            here = torch.cat([t[:n - first] > p - window if window else torch.ones(n - first, dtype=torch.bool), tree])
            if not here.any():
                continue
            x, y = kk[here], vv[here]  # [tokens, hk, d]
            for h in range(hk):
                rows = qq[i, h * g:(h + 1) * g]
                s = (rows @ x[:, h].T) * scale
                m = s.max(1, keepdim=True).values
                w = torch.exp(s - m)
                out[b, i, h * g:(h + 1) * g] = (w @ y[:, h]) / w.sum(1, keepdim=True)
                lse[b, i, h * g:(h + 1) * g] = (m + torch.log(w.sum(1, keepdim=True)))[:, 0]
                ds = (width + 4) * 2 * U * abs(scale) * (rows.abs() @ x[:, h].abs().T).amax(1) + 4 * U * s.abs().amax(1)
                steps = (int(here.sum()) + 64) * 2 * U
                split = 0.0 if q.dtype == torch.float32 else 2.0 ** -16
                tol[b, i, h * g:(h + 1) * g] = (2 * float(y[:, h].abs().max()) * (ds + 8 * U + steps + split))[:, None]
                ltol[b, i, h * g:(h + 1) * g] = 2 * (ds + 8 * U + steps) + 8 * U * lse[b, i, h * g:(h + 1) * g].abs()
    return out, lse, tol + final_round(out, q.dtype), ltol, live


def plan(parents, lens, table, page, pages, counts=None):
    """(mask, positions, slots) of rows of parents, every one as a whole sequence."""
    nodes = len(parents[0]) if parents else 0
    mask, pos, slots = [], [], []
    for b, row in enumerate(parents):
        n, c = lens[b], nodes if counts is None else counts[b]
        if not 0 <= c <= nodes or n < 0 or any(not -1 <= row[i] < i for i in range(c)):
            n, c = 0, 0
        sets = ancestors(row[:c]) + [set()] * (nodes - c)
        mask.append(words(sets, nodes))
        pos.append([n + len(s) - 1 if s else 0 for s in sets])
        got = []
        for i in range(nodes):
            col = (n + i) // page
            e = table[b][col] if i < c and col < len(table[b]) else -1
            got.append(e * page + (n + i) % page if 0 <= e < pages else -1)
        slots.append(got)
    return torch.stack(mask), torch.tensor(pos), torch.tensor(slots)


def pages_step(refs, table, lens, origin, keep, want, page, cols):
    """One step of the bookkeeping, row after row: (refs, table, lens, src, dst, rows, error)."""
    pool, up = len(refs), lambda x: -(-x // page)
    cnt, error = list(refs), 0
    lens = list(lens)
    for f, n in enumerate(lens):
        if not 0 <= n <= cols * page:
            lens[f], error = 0, 1
        for j in range(up(lens[f])):
            e = table[f][j]
            if 0 <= e < pool:
                cnt[e] -= 1
            else:
                error = 1
    rows = []
    for o, k, w in zip(origin, keep, want):
        most = lens[o] if 0 <= o < len(lens) else 0
        if not -1 <= o < len(lens) or not 0 <= k <= most or not k <= w <= cols * page:
            o, k, w, error = -1, 0, 0, 1
        held = [table[o][j] if 0 <= table[o][j] < pool else -1 for j in range(up(k))]
        error |= -1 in held
        for e in held:
            if e >= 0:
                cnt[e] += 1
        rows.append((k, w, held))
    free = [i for i, x in enumerate(cnt) if x == 0]
    total, after, out = 0, list(cnt), ([], [], [], [], [])
    for k, w, held in rows:
        copies = k % page != 0 and w > k and held[-1] >= 0 and cnt[held[-1]] > 1
        need = up(w) - up(k) + copies
        total += need
        served = need == 0 or total <= len(free)
        error |= 0 if served else 2
        line, src, dst, part = list(held), -1, -1, 0
        if served:
            fresh = free[total - need:total]
            for e in fresh:
                after[e] = 1
            if copies:
                src, dst, part = held[-1], fresh[0], k % page
                after[src] -= 1
                line = held[:-1]
            line += fresh
        for x, y in zip(out, (line + [-1] * (cols - len(line)), w if served else k, src, dst, part)):
            x.append(y)
    return (after,) + out + (error,)
