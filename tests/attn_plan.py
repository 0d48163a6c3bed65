"""How a one-token attention call is laid out over the GPU, restated from the rules that the
kernels' comments give: which way the work is shared out, and the bytes of workspace.

A pair is a key-value head with a block of at most `heads` query heads, of one sequence. Its
tokens go in rounds of four warps' tiles and in chunks of 128 tokens, or longer ones where
that would make too many. The ways:
    "one chunk"         no pair can have two chunks: no workspace
    "pair"              a CTA a pair: more chunks than resident CTAs, no pair over four rounds
    "chunk"             a CTA a chunk, a slot a pair; no headers
    "shares by pair"    shares of all the work, a slot and a header a pair
    "shares by CTA"     the same, a slot and a header a CTA
"""
from __future__ import annotations

SMS = 152


def plan(element_bytes, batch, kv_heads, group, head_dim, max_seen):
    """(way, slots, bytes of workspace)."""
    if element_bytes == 4:
        heads = 1 if group == 1 else 4 if group <= 4 else 8
    else:
        heads = 16 if group > 8 and head_dim <= 128 else 8
    dims = 64 if head_dim <= 64 else 128 if head_dim <= 128 else 256
    tile = min(32, 8192 // (dims * element_bytes))
    ctas = 2 if dims > 64 or element_bytes > 2 else 3 if heads > 8 else 4
    round_, resident = 4 * tile, SMS * ctas
    blocks = -(-group // heads)
    heads = min(heads, group)
    pairs_each = kv_heads * blocks
    rounds = -(-max_seen // round_)
    most = min(128, max(16, resident // pairs_each))
    chunks = min(most, -(-rounds // (128 // round_)))
    pairs = batch * pairs_each
    units = pairs * max(1, chunks)
    by_pair = pairs <= resident
    slots = 0 if chunks <= 1 else pairs if by_pair else resident
    four = lambda n: -(-n // 4) * 4  # noqa: E731
    size = 16 + 4 * (four(chunks * heads * 2) + four(chunks * heads * head_dim))
    if units > resident and pairs <= 3 * resident and rounds <= 4:
        way = "pair" if slots else "one chunk"
    elif not slots:
        way = "one chunk"
    elif units <= 3 * resident and by_pair:
        way = "chunk"
    else:
        way = "shares by pair" if by_pair else "shares by CTA"
    return way, slots, slots * size
