"""The decode-step operators from their definitions, in 64 bits on the CPU, and
how far a binary32 computation with one final rounding may be from them.

Bounds. u = 2^-24 is binary32's unit roundoff. Tensor-core accumulation is taken
as good to 2u a step (it may truncate), every other operation to u, exp and log to
4u. A score is a dot product of D terms, so it is off by at most
ds = (D + 4) 2u scale sum|q||k|, and a softmax weight by a factor 1 + ds + 8u. An
output sum of n weighted values passes through at most n / 16 + 64 roundings
(16 tokens a step, then the joins) and the weights may be held as two 16-bit
parts (2^-16), so with V = max |v| and twice for the quotient's two sides
    |o - exact| <= 2 V (ds + 8u + (n / 16 + 64) 2u + 2^-16 [16-bit types]) + r |exact|
where r is the type's unit roundoff (and half its smallest subnormal).
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -149), torch.bfloat16: (2.0 ** -8, 2.0 ** -133),
         torch.float16: (2.0 ** -11, 2.0 ** -24)}


def final_round(exact, dtype):
    r, tiny = ROUND[dtype]
    return r * exact.abs() + tiny


def decode(q, k, v, table, lens, scale, window=0):
    """(out, lse, out bound, lse bound); k, v [pages, page, heads, dim] on any device."""
    batch, hq, width = q.shape
    page, hk = k.shape[1], k.shape[2]
    out = torch.zeros((batch, hq, width), dtype=torch.float64)
    lse = torch.full((batch, hq), float("-inf"), dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(batch):
        n = int(lens[b])
        t = torch.arange(max(0, n - window) if window else 0, n)
        if not len(t):
            continue
        pages = table[b].cpu().long()[t // page]
        at = (pages.to(k.device), (t % page).to(k.device))
        kk, vv = k[at].double().cpu(), v[at].double().cpu()
        for h in range(hq):
            x, y, z = q[b, h].double().cpu(), kk[:, h * hk // hq], vv[:, h * hk // hq]
            s = (y @ x) * scale
            m = s.max()
            p = torch.exp(s - m)
            out[b, h] = (p @ z) / p.sum()
            lse[b, h] = m + torch.log(p.sum())
            ds = (width + 4) * 2 * U * abs(scale) * float((y.abs() @ x.abs()).max())
            steps = (len(t) / 16 + 64) * 2 * U
            split = 0.0 if q.dtype == torch.float32 else 2.0 ** -16
            tol[b, h] = 2 * float(z.abs().max()) * (ds + 8 * U + steps + split)
            ltol[b, h] = 2 * (ds + 8 * U + steps) + 8 * U * abs(float(lse[b, h]))
    return out, lse, tol + final_round(out, q.dtype), ltol


def rotate(x, cos_sin, positions, rot, interleaved):
    """(rotated x in 64 bits, bound): two products and a sum in binary32, one rounding."""
    y = x.double().cpu().clone()
    cs = cos_sin.double().cpu()[positions.cpu()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    ia = torch.arange(rot // 2) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    tol = torch.zeros_like(y)
    tol[..., ia] = tol[..., ib] = 3 * U * (a.abs() + b.abs())
    return y, tol + final_round(y, x.dtype)


def join(parts, lses):
    """(out, lse, out bound, lse bound) of W ranks' parts; bounds as above with W steps."""
    lse_r = torch.stack([x.double().cpu() for x in lses])
    m = lse_r.amax(0)
    base = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    w = torch.exp(lse_r - base)
    total = w.sum(0)
    out, big = torch.zeros(parts[0].shape, dtype=torch.float64), torch.zeros(parts[0].shape[:-1], dtype=torch.float64)
    for part, x in zip(parts, w):
        y = torch.where((x > 0)[..., None], part.double().cpu(), 0.0)
        out += y * x[..., None]
        big = torch.maximum(big, y.abs().amax(-1))
    out /= torch.where(total == 0, torch.ones_like(total), total)[..., None]
    lse = base + torch.log(total)
    # a weight is off by u of the difference of two lses (each exact), then exp's 4u
    spread = torch.where(w > 0, (lse_r - base).abs(), torch.zeros_like(w)).amax(0)
    rel = (spread + 8 + 2 * len(parts)) * 2 * U
    tol = 2 * (big * rel)[..., None] + final_round(out, parts[0].dtype)
    ltol = 2 * rel + 8 * U * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())
    return out, lse, tol, ltol


def assert_near(got, want, tol, what):
    """Within tol where `want` is finite, equal (or both NaN) elsewhere."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    fine = torch.isfinite(want)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(same[~fine].all()), f"{what}: a value that is not finite differs"
    off = torch.where(fine, (got - want).abs() - tol, torch.zeros_like(want))
    assert not bool(torch.isnan(got[fine]).any()), f"{what}: NaN"
    assert float(off.max() if off.numel() else 0.0) <= 0.0, (
        f"{what}: {int((off > 0).sum())} of {off.numel()} values off by more than their bound, by up to "
        f"{float(off.max()):.3g}")
