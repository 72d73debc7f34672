"""Plain 64-bit reference of the 4-bit paged cache (include/fk_kv4.h), from
the definitions, on the CPU.  Shares nothing with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def codebook(H, seed=0, spread=0.02):
    g = torch.Generator().manual_seed(seed)
    u = torch.linspace(-1, 1, 16) * 0.97
    c = u.sign() * u.abs() ** 1.25 + spread * torch.randn(2, H, 16, generator=g)
    return c.clamp(-1, 1).sort(-1).values.half()


def place(D, kv, t, d):
    """(byte, shift) of the code of token t (< 32), dimension d in a block."""
    if kv == 0:
        lane = 16 * (d // (D // 4)) + 4 * (t // 8) + t % 4
        w = d % (D // 4)
        a = (t // 4 % 2) * (D // 8) + w // 2
    else:
        lane = 16 * (t // 8) + d // (D // 16)
        w = d % (D // 16)
        a = 32 * (w // 8) + (t % 8) * min(4, D // 32) + w % 8 // 2
    return 1024 * (a // 16) + 16 * lane + a % 16, 4 * (d % 2)


def place_tables(D, kv):
    at = np.array([[place(D, kv, t, d) for d in range(D)] for t in range(32)])
    return torch.from_numpy(at[..., 0]), torch.from_numpy(at[..., 1])


def encode(x, cb):
    """Rows x (T, H, D) of a 16-bit type, cb (H, 16): codes, scales (float64)."""
    x = x.double()
    s = x.abs().amax(-1)
    s = torch.where(torch.isfinite(x).all(-1), s, math.nan)
    t = ((cb[:, :-1].double() + cb[:, 1:].double()) / 2).half().double()
    code = (t[None, :, None, :] * s[..., None, None] < x[..., None]).sum(-1)
    return code.to(torch.uint8), s


def gather(codes, scales, cb, page, tok):
    """Values (2, n, H, D) in float64 of tokens tok (n) of pages page (n)."""
    H, D = codes.shape[1], codes.shape[4] // 16
    out = []
    for kv in (0, 1):
        at, sh = place_tables(D, kv)
        rows = codes[page, :, kv, tok // 32]                       # (n, H, 16 D)
        b = torch.gather(rows, 2, at[tok % 32][:, None].expand(-1, H, -1))
        c = (b.int() >> sh[tok % 32][:, None]) & 15
        v = torch.gather(cb[kv].double()[None].expand(len(page), -1, -1), 2, c.long())
        out.append(v * scales[page, :, kv, tok].double()[..., None])
    return torch.stack(out)


def plan(ctx, new, P, table, free, count, cap):
    """The step's plan, request by request; table (list of lists) is changed."""
    ctx, new = [max(0, c) for c in ctx], [max(0, n) for n in new]
    n = min(max(count, 0), len(free))
    M, left, wanted, lost = len(table[0]), n, 0, 0
    slots, pos, cu = [], [], [0]
    for b, (c, f) in enumerate(zip(ctx, new)):
        held = -(-c // P)
        for p in range(held, min(-(-(c + f) // P), M)):
            wanted += 1
            table[b][p] = free[left - 1] if left > 0 else -1
            left -= left > 0
        got = 0
        for p in range(held, M):
            got += p < -(-(c + f) // P) and table[b][p] >= 0
        end = (min(held, M) + got) * P
        lost += max(0, c + f - max(c, end))
        for i in range(c, c + f):
            page = table[b][i // P] if i // P < M else -1
            slots.append(page * P + i % P if page >= 0 else -1)
            pos.append(i)
        cu.append(cu[-1] + f)
    total = cu[-1]
    slots, pos = slots[:cap], pos[:cap]
    slots += [-1] * (cap - len(slots))
    pos += [-1] * (cap - len(pos))
    return dict(seq=[c + f for c, f in zip(ctx, new)], cu=cu, slots=slots, pos=pos, left=left,
                status=[total, n - left, wanted - (n - left), lost])


def attention(q, cu, seq, table, cb, codes, scales, scale, causal, window):
    """out, lse, and what bounds the error: sum of p |v|, of |q k|, the keys."""
    T, Hq, D = q.shape
    H, P, pages = codes.shape[1], scales.shape[3], codes.shape[0]
    G = Hq // H
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    pv, dot = torch.zeros_like(out), torch.zeros_like(lse)
    svmax = torch.zeros_like(lse)
    M = table.shape[1]
    for b in range(len(seq)):
        n, S = int(cu[b + 1] - cu[b]), int(seq[b])
        j = torch.arange(min(S, M * P))
        page = table[b].long()[j // P]
        ok = (page >= 0) & (page < pages)
        j, page = j[ok], page[ok]
        if n == 0 or len(j) == 0:
            continue
        k, v = gather(codes, scales, cb, page, j % P)              # (n, H, D)
        at = slice(int(cu[b]), int(cu[b + 1]))
        x = q[at].double().view(n, H, G, D)
        pos = torch.arange(S - n, S)[:, None]
        seen = torch.ones(n, len(j), dtype=torch.bool)
        if causal:
            seen &= j <= pos
        if window:
            seen &= j > pos - window
        s = torch.einsum("nhgd,shd->nhgs", x, k) * scale
        s = torch.where(seen[:, None, None], s, -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.where(seen[:, None, None], torch.exp(s - torch.where(top > -math.inf, top, 0.0)), 0.0)
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l == 0, 1.0, l)
        vz = torch.where(seen.any(0)[:, None, None], v, 0.0)       # what no row sees counts for nothing
        out[at] = torch.einsum("nhgs,shd->nhgd", p, vz).reshape(n, Hq, D)
        # a key some rows see and others do not: 0 * NaN must not spread
        if not torch.isfinite(vz).all():
            for i in range(n):
                w = torch.where(seen[i][:, None, None], v, 0.0)
                out[at][i] = torch.einsum("hgs,shd->hgd", p[i], w).reshape(Hq, D)
        lse[at] = (top + torch.log(l))[..., 0].reshape(n, Hq)
        # bounds of the error count finite values only (rows that see others are NaN)
        p, k, vz = (torch.nan_to_num(t, 0.0, 0.0, 0.0) for t in (p, k, vz))
        pv[at] = torch.einsum("nhgs,shd->nhgd", p, vz.abs()).reshape(n, Hq, D)
        dot[at] = (torch.einsum("nhgd,shd->nhgs", x.abs(), k.abs()) * scale * seen[:, None, None]
                   ).amax(-1).reshape(n, Hq)
        svmax[at] = (vz.abs().amax(-1).amax(0)[:, None] * torch.ones(G)).reshape(Hq) * len(j)
    return out, lse, pv, dot, svmax


def attention_tolerance(out, lse, pv, dot, svmax, D, dtype):
    """Largest errors that the kernel's roundings allow.

    Scores: products of two fp16 numbers are exact, D of them are added in
    fp32 and three more factors follow: |ds| <= (D + 4) 2^-24 dot, plus an
    exponential good to 2^-22 relative.  A weight is rounded to fp16 once:
    2^-11 of p |v|, or 2^-25 of the largest v scale for each key where that
    is more (weights are at most 64 times the scale's unit, sums at least 1).
    Sums over the keys are fp32.  The result is rounded to its type."""
    ds = (D + 4) * 2.0 ** -24 * dot + 2.0 ** -21
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-38
    tol = u * out.abs() + (2.0 ** -11 + 2 * ds + 2.0 ** -16)[..., None] * pv
    tol = tol + (2.0 ** -25 * svmax)[..., None] + tiny
    return tol, 2 * ds + 2.0 ** -20 * torch.where(torch.isfinite(lse), lse.abs(), 0.0) + 2.0 ** -20
