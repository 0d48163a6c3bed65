"""One decode step of W tensor-parallel ranks on one device, from the new token's
projection to the joined hidden state.

Each rank holds its own heads' part of a paged key-value cache and of the output
projection. Per step, and per rank:

  1. ``detfold_kv_append``    rotates the new tokens' keys and queries and appends
                              keys and values to the rank's cache;
  2. ``detfold_attn_decode``  attends over the rank's cache, one new token a sequence;
  3. a matrix product         projects the rank's heads to a hidden-size partial sum;

then ``detfold_loopback_allreduce`` folds the W partial sums in ascending rank order, so
that every rank holds the same bits. ``sequence_parallel`` shows the other way to split a
cache, by tokens: each rank attends to its own pages and ``detfold_attn_join`` joins the ranks'
partial attentions in rank order.

Run it as ``python examples/decode_step.py``; it prompts a small random model's one layer,
decodes a few steps and checks them against a plain computation in 64 bits.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_fixed_order_gb300 as df  # noqa: E402


def rotation_table(positions: int, rot_dim: int, device="cuda") -> torch.Tensor:
    """cos then sin of p / 10000^(2i / rot_dim), as ``df.Rope`` takes them."""
    freq = 10000.0 ** (-torch.arange(rot_dim // 2, dtype=torch.float64, device=device) * 2 / rot_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Rank:
    """One rank's heads: its cache, its slice of the projections and its buffers."""

    def __init__(self, wqkv, wo, q_heads, kv_heads, head_dim, pages, page_size, batch, max_len, rope, dtype):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.wqkv, self.wo, self.rope, self.max_len = wqkv, wo, rope, max_len
        shape = (pages, page_size, kv_heads, head_dim)
        self.cache = df.PagedCache(torch.zeros(shape, dtype=dtype, device="cuda"),
                                   torch.zeros(shape, dtype=dtype, device="cuda"))
        self.attended = torch.empty((batch, q_heads, head_dim), dtype=dtype, device="cuda")
        need = df.detfold_attn_decode_workspace_bytes(self.cache, batch, q_heads, max_len)
        self.workspace = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def append(self, x, slots, positions):
        """Projects x [tokens, hidden], appends its keys and values, returns its rotated queries."""
        qkv = (x @ self.wqkv).view(x.shape[0], self.q_heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        df.detfold_kv_append(self.cache, k, v, slots, rope=self.rope, positions=positions, q=q, q_out=q)
        return q

    def step(self, x, slots, positions, table, lens):
        """This rank's partial sum of the layer's output, [batch, hidden] float32."""
        q = self.append(x, slots, positions)
        df.detfold_attn_decode(self.attended, q, self.cache, table, lens, self.max_len, self.head_dim ** -0.5,
                               workspace=self.workspace)
        return self.attended.view(x.shape[0], -1).float() @ self.wo.float()


def tensor_parallel(ranks, x, slots, positions, table, lens):
    """The layer's output after one step: W ranks' partial sums, folded in rank order."""
    partial = [r.step(x, slots, positions, table, lens) for r in ranks]
    df.loopback_allreduce([p.view(-1) for p in partial])
    return partial


def sequence_parallel(q, cache, page_size, tables, lens, scale):
    """Attention of q over a cache whose pages W ranks share out: tables[r] and lens[r] are
    rank r's pages and tokens of each sequence. Returns (out, lse)."""
    parts, lses = [], []
    for table, n in zip(tables, lens):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)
        max_len = table.shape[1] * page_size
        need = df.detfold_attn_decode_workspace_bytes(cache, q.shape[0], q.shape[1], max_len)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
        df.detfold_attn_decode(out, q, cache, table, n, max_len, scale, lse=lse, workspace=ws)
        parts.append(out)
        lses.append(lse)
    out, lse = torch.empty_like(q), torch.empty_like(lses[0])
    df.detfold_attn_join(out, parts, lses, lse=lse)
    return out, lse


def plain_layer(history, wqkv, wo, q_heads, kv_heads, head_dim, cos_sin):
    """The last token's output of one sequence in 64 bits; history [tokens, hidden]."""
    x = history.double()
    qkv = (x @ wqkv.double()).view(len(x), q_heads + 2 * kv_heads, head_dim)
    q, k, v = qkv.split([q_heads, kv_heads, kv_heads], 1)
    half = cos_sin.shape[1] // 2
    cos, sin = cos_sin.double()[:len(x), None, :half], cos_sin.double()[:len(x), None, half:]

    def turn(y):
        a, b = y[..., :half], y[..., half:2 * half]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * half:]], -1)

    q, k = turn(q)[-1], turn(k).repeat_interleave(q_heads // kv_heads, 1)
    v = v.repeat_interleave(q_heads // kv_heads, 1)
    p = torch.softmax(torch.einsum("hd,thd->ht", q, k) * head_dim ** -0.5, -1)
    return torch.einsum("ht,thd->hd", p, v).reshape(-1) @ wo.double()


def main(world=2, hidden=512, q_heads=8, kv_heads=4, head_dim=64, page_size=16, prompts=(37, 5, 120), steps=4, seed=0,
         dtype=torch.bfloat16):
    """Prompts, decodes `steps` tokens on `world` ranks, returns the largest relative error of a step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    batch, longest = len(prompts), max(prompts) + steps
    cols = -(-longest // page_size)
    rope_table = rotation_table(longest, head_dim)
    rope = df.Rope(rope_table)
    qh, kh = q_heads // world, kv_heads // world
    make = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[0] ** -0.5).to(dtype)  # noqa: E731
    wqkv = [make(hidden, (qh + 2 * kh) * head_dim) for _ in range(world)]
    wo = [make(qh * head_dim, hidden) for _ in range(world)]
    ranks = [Rank(wqkv[r], wo[r], qh, kh, head_dim, batch * cols, page_size, batch, longest, rope, dtype)
             for r in range(world)]
    table = torch.randperm(batch * cols, generator=g, device="cuda").to(torch.int32).view(batch, cols)

    def slots_of(b, positions):
        return table[b, positions // page_size].long() * page_size + positions % page_size

    history = []
    for b, n in enumerate(prompts):  # prompts: many tokens at once
        x = torch.randn((n, hidden), generator=g, device="cuda").to(dtype)
        positions = torch.arange(n, device="cuda")
        for r in ranks:
            r.append(x, slots_of(b, positions), positions)
        history.append(x)
    worst = 0.0
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    rows = torch.arange(batch, device="cuda")
    for _ in range(steps):
        x = torch.randn((batch, hidden), generator=g, device="cuda").to(dtype)
        positions = lens.long()
        lens = lens + 1
        outs = tensor_parallel(ranks, x, slots_of(rows, positions), positions, table, lens)
        assert all(torch.equal(o, outs[0]) for o in outs), "every rank holds the same bits"
        history = [torch.cat([h, x[b:b + 1]]) for b, h in enumerate(history)]
        for b in range(batch):
            want = sum(plain_layer(history[b], wqkv[r], wo[r], qh, kh, head_dim, rope_table) for r in range(world))
            worst = max(worst, float((outs[0][b] - want).norm() / want.norm()))

    # the same cache shared out by pages: rank r attends to every world-th page of each sequence
    q = torch.randn((batch, qh, head_dim), generator=g, device="cuda").to(dtype)
    whole, lse = torch.empty_like(q), torch.empty((batch, qh), device="cuda")
    df.detfold_attn_decode(whole, q, ranks[0].cache, table, lens, longest, head_dim ** -0.5, lse=lse,
                           workspace=ranks[0].workspace)
    tables, parts = [], []
    for r in range(world):
        mine = table[:, r::world].contiguous()
        starts = torch.arange(r, cols, world, device="cuda") * page_size
        tables.append(mine)
        parts.append((lens[:, None] - starts).clamp(0, page_size).sum(1).to(torch.int32))
    joined, joined_lse = sequence_parallel(q, ranks[0].cache, page_size, tables, parts, head_dim ** -0.5)
    apart = float((joined.float() - whole.float()).norm() / whole.float().norm())
    assert torch.allclose(joined_lse, lse, atol=1e-4), "the joined log-sums are the whole's"
    return worst, apart


if __name__ == "__main__":
    error, apart = main()
    print(f"decode steps: relative error {error:.2e} against 64 bits; "
          f"sequence-parallel attention differs from the whole by {apart:.2e}")
