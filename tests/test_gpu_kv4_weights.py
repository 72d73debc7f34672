"""Attention over the 4-bit cache where v scales differ by many orders of
magnitude: what a row adds up must keep its bits whatever the scales of tokens
that it hardly counts, or that only another row of its tile sees."""
import math

import numpy as np
import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref

pytestmark = pytest.mark.gpu
DT = ref.DT


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def definition(q, cu, seq, table, cb, codes, scales, scale, causal, window):
    """out and lse in 64 bits; sum of p |v| and the largest |q k|; each row's
    largest p_j * v scale and the number of keys it sees."""
    T, Hq, D = q.shape
    H, P = codes.shape[1], scales.shape[3]
    G = Hq // H
    out, pv = (torch.zeros(T, Hq, D, dtype=torch.float64) for _ in range(2))
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    dot, top, keys = (torch.zeros(T, Hq, dtype=torch.float64) for _ in range(3))
    for b, S in enumerate(seq):
        n = int(cu[b + 1] - cu[b])
        j = torch.arange(S)
        page = table[b].long()[j // P]
        k, v = ref.gather(codes, scales, cb, page, j % P)
        vs = scales[page, :, 1, j % P].double()                    # (S, H)
        at = slice(int(cu[b]), int(cu[b]) + n)
        pos = torch.arange(S - n, S)[:, None]
        see = torch.ones(n, S, dtype=torch.bool)
        see &= j <= pos if causal else True
        see &= j > pos - window if window else True
        see = see[None, :, None]                                   # (1, n, 1, S)
        x = q[at].double().view(n, H, G, D).transpose(0, 1).reshape(H, n * G, D)
        k, v = k.transpose(0, 1), v.transpose(0, 1)                # (H, S, D)
        s = (x @ k.transpose(1, 2).contiguous() * scale).view(H, n, G, S).masked_fill(~see, -math.inf)
        l = torch.logsumexp(s, -1, keepdim=True)
        p = torch.exp(s - torch.where(l > -math.inf, l, 0.0))

        def rows(t):                                               # (H, n, G, ...) -> (n, Hq, ...)
            return t.transpose(0, 1).reshape(n, Hq, *t.shape[3:])
        out[at], pv[at] = (rows((p.view(H, n * G, S) @ w).view(H, n, G, D)) for w in (v, v.abs()))
        lse[at] = rows(l[..., 0])
        dot[at] = rows(((x.abs() @ k.abs().transpose(1, 2).contiguous()).view(H, n, G, S) * see).amax(-1)) * scale
        top[at] = rows((p * vs.T[:, None, None]).amax(-1))
        keys[at] = rows(see.sum(-1).expand(H, n, G).double())
    return out, lse, pv, dot, top, keys


def tolerance(want, D, dtype, cmax):
    """Scores, exponentials and sums as in the plain tests' bounds.  A weight
    is rounded to fp16 once: 2^-11 of itself, or, below fp16's normal range,
    2^-25 where the row's largest weight is 4 at least (it is set to 8 by
    logarithms good to a few units): 2^-27 of the row's largest p * v scale,
    for each key, times the largest codebook value."""
    out, lse, pv, dot, top, keys = want
    ds = (D + 4) * 2.0 ** -24 * dot + 2.0 ** -21
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-38
    tol = u * out.abs() + (2.0 ** -11 + 2 * ds + 2.0 ** -16)[..., None] * pv
    tol = tol + (2.0 ** -27 * keys * top * cmax)[..., None] + tiny
    return tol, 2 * ds + 2.0 ** -20 * torch.where(torch.isfinite(lse), lse.abs(), 0.0) + 2.0 ** -20


def run(seq, qlen, Hq, H, D, P, dtype, setup, causal=True, window=0, extra=0, seed=0):
    """setup(codes, scales, at) changes the cache; at(b, j) is (page, place)."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-s // P) for s in seq]
    M, pages = max(held) + extra, sum(held) + 1
    table = torch.full((len(seq), M), -1, dtype=torch.int32)
    ids, used = torch.randperm(pages, generator=g).int(), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[used:used + n]
        used += n
    codes = torch.randint(0, 256, (pages, H, 2, P // 32, 16 * D), dtype=torch.uint8, generator=g)
    scales = torch.ones(pages, H, 2, P).to(DT[dtype])
    scales[:, :, 0] = 0                                            # equal scores
    cb = ref.codebook(H, seed)
    setup(codes, scales, lambda b, j: (table[b].long()[j // P], j % P))
    cu = torch.tensor([0] + list(np.cumsum(qlen)), dtype=torch.int32)
    T = int(cu[-1])
    q = torch.ones(T, Hq, D, dtype=DT[dtype])
    out = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    scale = 1 / math.sqrt(D)
    dev = [t.cuda() for t in (q, cu, torch.tensor(seq, dtype=torch.int32), table, cb, codes, scales)]
    fk.fk_kv4_attention(*dev, out, max(qlen), scale=scale, causal=causal, window=window, lse=lse)
    want = definition(q, cu, seq, table, cb, codes, scales, scale, causal, window)
    tol, tol_lse = tolerance(want, D, DT[dtype], float(cb.abs().max()))
    err, e = (out.cpu().double() - want[0]).abs(), (lse.cpu().double() - want[1]).abs()
    assert bool((err <= tol).all()), f"out: {float((err / tol).max())} times the tolerance"
    ok = torch.isfinite(want[1])
    assert bool((e <= tol_lse)[ok].all()), f"lse: {float((e / tol_lse)[ok].max())} times the tolerance"


def outlier(j, big, weightless=True):
    """Token j of request 0 has a v scale of `big` and, weightless, a score far
    below the others': codes of the lowest value under a large k scale."""
    def setup(codes, scales, at):
        page, i = at(0, torch.tensor(j))
        scales[page, :, 1, i] = big
        if weightless:
            D = codes.shape[4] // 16
            by, _ = ref.place_tables(D, 0)
            codes[page, :, 0, i // 32][:, by[i % 32]] = 0          # both nibbles: the dimension and its neighbour
            scales[page, :, 0, i] = 64.0
    return setup


# a token of no weight first, in the middle, and last but one, in every form:
# one and several waves of a group, shares with a join, rows; several row tiles
FORMS = [dict(seq=[600], qlen=[1], Hq=4, H=1), dict(seq=[600], qlen=[1], Hq=4, H=1, extra=200),
         dict(seq=[600, 70], qlen=[30, 3], Hq=4, H=1), dict(seq=[600, 70], qlen=[30, 3], Hq=4, H=1, extra=200),
         dict(seq=[600] + [64] * 129, qlen=[1] * 130, Hq=8, H=8)]


@pytest.mark.parametrize("dtype,big,rest", [("bf16", 2.0 ** 26, 1.0), ("bf16", 1000.0, 1.0), ("f16", 32768.0, 2.0 ** -9)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_a_weightless_token_of_a_large_scale(form, D, dtype, big, rest):
    for j in (0, 300, 566):
        def setup(codes, scales, at):
            scales[:, :, 1] = rest
            outlier(j, big)(codes, scales, at)
        run(D=D, P=32, dtype=dtype, setup=setup, seed=form, **FORMS[form])


@pytest.mark.parametrize("dtype,big,rest", [("bf16", 2.0 ** 26, 1.0), ("f16", 32768.0, 2.0 ** -9)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 48])
def test_a_large_scale_that_other_rows_of_the_tile_see(window, D, dtype, big, rest):
    # the later rows see it under the causal mask, the earlier ones under the window
    for j in (590, 540):
        def setup(codes, scales, at):
            scales[:, :, 1] = rest
            outlier(j, big, weightless=False)(codes, scales, at)
        for extra in (0, 200):
            run([600], [24], 2, 1, D, 32, dtype, setup, window=window, extra=extra, seed=D)


@pytest.mark.parametrize("dtype,big,rest", [("bf16", 2.0 ** 26, 1.0), ("f16", 32768.0, 2.0 ** -9)])
@pytest.mark.parametrize("D,H", [(64, 110), (128, 90), (256, 32)])
@pytest.mark.parametrize("window", [0, 20])
def test_a_large_scale_among_prompts_that_fill_the_card(window, D, H, dtype, big, rest):
    for weightless in (False, True):
        def setup(codes, scales, at):
            scales[:, :, 1] = rest
            outlier(40, big, weightless)(codes, scales, at)
        run([90], [90], 12 * H, H, D, 32, dtype, setup, window=window, seed=2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("extra", [0, 200])
def test_scales_that_rise_and_fall(dtype, extra):
    # every token another magnitude, runs of zeros first and last: l alone grows there
    def setup(codes, scales, at):
        g = torch.Generator().manual_seed(1)
        page, i = at(0, torch.arange(900))
        e = torch.randint(-12, 13, (900,), generator=g) if dtype == "f16" else torch.randint(-80, 30, (900,), generator=g)
        v = torch.exp2(e.float())
        v[:100] = 0
        v[-40:] = 0
        scales[page, :, 1, i] = v.to(scales.dtype)[:, None]
        scales[page, :, 0, i] = torch.rand(900, generator=g).to(scales.dtype)[:, None]
    for D in (64, 128, 256):
        run([900], [3], 4, 2, D, 32, dtype, setup, extra=extra, seed=5)
