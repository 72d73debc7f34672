"""Plain references of the operators around a serving step (include/fk_serve.h),
from their definitions, on the CPU.  Share nothing with the library."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np
import torch


# ---- rotary positions ----------------------------------------------------------

def frequencies(R, base=10000.0, stretch=1.0, trained=0, slow=1.0, fast=32.0):
    w = np.array([base ** (-2 * i / R) for i in range(R // 2)])
    share = np.clip((trained * w / (2 * math.pi) - slow) / (fast - slow), 0, 1) if trained else np.zeros(R // 2)
    return share * w + (1 - share) * w / stretch


def rope(x, pos, w, interleaved=False, inverse=False, factor=1.0):
    """x (T, H, D) -> float64."""
    x = x.double().cpu()
    R = 2 * len(w)
    y = x.clone()
    for t, p in enumerate(pos):
        if p < 0:
            continue
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            th = float(p) * float(w[i]) * (-1 if inverse else 1)
            c, s = math.cos(th), math.sin(th)
            y[t, :, a] = factor * (x[t, :, a] * c - x[t, :, b] * s)
            y[t, :, b] = factor * (x[t, :, a] * s + x[t, :, b] * c)
    return y


def rope_tolerance(x, y, w, pos, interleaved, factor, dtype):
    """Errors that the roundings allow.  Angle: the table's entry is off by
    2^-53 of w and the reference's product by as much of the angle, so 2 p w
    2^-53; the fraction of a turn by 2^-33 turn.  The octant's angle (up to
    0.79) is rounded three times in fp32, the series end below 3e-9 and their
    last steps round to 2^-24: 6 2^-24 for a sine or cosine in all, times the
    factor, rounded.  Products and their sum: two more roundings.  The result
    is rounded to its type, below its normal values to their last place."""
    x = x.double().cpu().abs()
    R, u = 2 * len(w), torch.finfo(dtype).eps / 2
    tol = torch.zeros_like(y)
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        far = torch.tensor([max(p, 0) * float(w[i]) for p in pos])
        e = (abs(factor) * (10 * 2.0 ** -24 + far * 2.0 ** -52))[:, None]
        tol[..., a] = tol[..., b] = e * (x[..., a] + x[..., b])
    tiny = torch.finfo(dtype).smallest_normal * u
    tol = torch.where(tol > 0, tol + u * y.abs() + tiny, tol)
    tol[[p < 0 for p in pos]] = 0
    return tol


# ---- verification ------------------------------------------------------------------

def weight(x):
    """floor(x 2^42) of a value clamped to 0 .. 1; NaN: 0."""
    x = float(x)
    return 0 if not x > 0 else int(math.floor(Fraction(min(x, 1.0)) * 2 ** 42))


def verify(cu, tokens, p, q, u, pick, seq):
    """accepted, emitted (by row; rows of no request absent), keep."""
    p = p.float().cpu().numpy()
    q = None if q is None else q.float().cpu().numpy()
    V = p.shape[1]
    accepted, emitted, keep = [], {}, []
    for b in range(len(cu) - 1):
        rows = range(cu[b], cu[b + 1])
        if not len(rows):
            accepted.append(0)
            keep.append(seq[b])
            continue
        best = {r: max(range(V), key=lambda i: (p[r][i] if p[r][i] == p[r][i] else -math.inf, -i)) for r in rows} if u is None else None
        n = 0
        while n < len(rows) - 1:
            r = rows[n]
            d = tokens[r + 1]
            if not 0 <= d < V:
                break
            if u is None:
                good = best[r] == d
            else:
                x, y = float(p[r][d]), 1.0 if q is None else float(q[r][d])
                good = (math.isfinite(x) and math.isfinite(y) and Fraction(float(u[r])) * Fraction(y) < Fraction(x)) or (
                    x == math.inf and y == y and y < math.inf)
            if not good:
                break
            n += 1
        r = rows[n]
        if u is None:
            token = best[r]
        else:
            plain = [weight(x) for x in p[r]]
            w = plain
            if n < len(rows) - 1:
                if q is None:
                    w = [0 if i == tokens[r + 1] else x for i, x in enumerate(plain)]
                else:
                    with np.errstate(invalid="ignore"):
                        w = [weight(x) for x in p[r] - q[r]]
                w = w if sum(w) else plain
            total, token = sum(w), -1
            if total:
                s = float(pick[b])
                s = min(max(s, 0.0), 1.0) if s == s else 0.0
                k = min(int(math.floor(Fraction(s) * 2 ** 31)), 2 ** 31 - 1)
                point, upto = k * total // 2 ** 31, 0
                for token, x in enumerate(w):
                    upto += x
                    if upto > point:
                        break
        accepted.append(n)
        keep.append(seq[b] - (len(rows) - 1 - n))
        for i, r in enumerate(rows):
            emitted[r] = tokens[r + 1] if i < n else token if i == n else -1
    return accepted, emitted, keep


# ---- pages -------------------------------------------------------------------------

class Pool:
    """Rows as lists of pages, the list, shares as counted from the rows."""

    def __init__(self, table, lens, free, pages, P, seq=None):
        self.table, self.lens, self.free, self.pages, self.P = [list(r) for r in table], list(lens), list(free), pages, P
        self.seq = list(seq) if seq is not None else None

    def held(self, r):
        return -(-self.lens[r] // self.P)

    def holders(self):
        n = [0] * self.pages
        for r in range(len(self.table)):
            for p in self.table[r][:self.held(r)]:
                n[p] += 1
        return n

    def shares(self):
        return [max(0, n - 1) for n in self.holders()]

    def fork(self, rows, sources, keep):
        R, P = len(self.table), self.P
        old, lens, refs = [list(r) for r in self.table], list(self.lens), self.holders()
        jobs = []
        for i, r in enumerate(rows):
            if not 0 <= r < R or r in rows[:i]:
                continue
            s = r if sources is None else sources[i]
            most = min(k for x, k in zip(rows, keep) if x == r)
            n = min(max(0, most), lens[s]) if 0 <= s < R else 0
            if s == r and n == lens[r]:
                continue
            jobs.append((i, r, s, n, -(-lens[r] // P)))
        order = []                                                # pages that are given up, in order
        for _, r, _, _, held in jobs:
            for p in old[r][:held]:
                refs[p] -= 1
                order.append(p)
        for _, _, s, n, _ in jobs:
            for p in old[s][:n // P] if n else []:
                refs[p] += 1
        goes_on, copy = {}, []
        for i, r, s, n, _ in jobs:
            if n % P:
                p = old[s][n // P]
                if refs[p] == 0 and p not in goes_on.values():
                    goes_on[i] = p
                else:
                    copy.append((i, p, n % P))
        for p in dict.fromkeys(order):
            if refs[p] == 0 and p not in goes_on.values():
                self.free.append(p)
        got = min(len(copy), len(self.free))
        taken = self.free[len(self.free) - got:]
        self.free = self.free[:len(self.free) - got]
        copies = [[-1, -1, 0] for _ in rows]
        for (i, p, t), to in zip(copy, taken):
            copies[i] = [p, to, t]
            goes_on[i] = to
        for i, r, s, n, held in jobs:
            whole = old[s][:n // P] if n else []
            end = [goes_on[i]] if i in goes_on else []
            self.lens[r] = n if end else n // P * P
            row = whole + end
            upto = max(held, n // P + 1)
            row += [-1] * (upto - len(row))
            self.table[r] = (row + old[r][len(row):])[:len(old[r])]
            if self.seq is not None:
                self.seq[r] = self.lens[r]
        return copies

    def compact(self):
        """moves; the pool with its new numbers."""
        free = set(self.free)
        used = self.pages - len(free)
        movers = [p for p in range(used, self.pages) if p not in free]
        holes = [p for p in range(used) if p in free]
        to = dict(zip(movers, holes))
        for r in range(len(self.table)):
            for e in range(self.held(r)):
                self.table[r][e] = to.get(self.table[r][e], self.table[r][e])
        self.free = list(range(self.pages - 1, used - 1, -1))
        return [[a, b, self.P] for a, b in zip(movers, holes)]
