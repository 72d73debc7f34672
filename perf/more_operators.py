"""More operators of a serving step on the paged 4-bit cache, as they are
measured: rotary positions before rows are appended, attention of requests
that share a prefix, verification of drafted tokens, and the pages of a cache
forked, returned, copied and compacted.

The cache is that of include/fk_kv4.h: blocks of 32 tokens of 4-bit codes with
one scale a row, pages of some blocks, a block table with a row of pages for
each request, a list of free pages.  A page that several rows hold counts them
in `shares`: holders beyond the first.
"""
import math
import random

import numpy as np
import torch

own = False                               # whether run() makes the package's calls; it is imported only there

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # queries and keys of one decode step, slices of the fused projection
        dict(name="rope decode 64", kind="rope", T=64, Hq=32, Hkv=8, D=128, R=128, dtype="bf16", interleaved=False, inverse=False,
             far=8000, stretch=1.0),
        # a prompt's tokens in a context stretched 32-fold
        dict(name="rope prompt 16384", kind="rope", T=16384, Hq=32, Hkv=8, D=128, R=128, dtype="bf16", interleaved=False, inverse=False,
             far=130000, stretch=32.0),
        # gradients in 32 bits: pairs side by side, half of the head, odd number of tokens
        dict(name="rope gradient 5001", kind="rope", T=5001, Hq=6, Hkv=3, D=64, R=32, dtype="f32", interleaved=True, inverse=True,
             far=6000, stretch=1.0),
        # one chat that drafts four tokens
        dict(name="verify one", kind="verify", B=1, n=5, V=32000, dtype="f32", draft=True, greedy=False),
        # a server's batch that drafts up to five tokens with a small model
        dict(name="verify 64", kind="verify", B=64, n=6, V=128000, dtype="f32", draft=True, greedy=False),
        # the most likely token is taken: drafts looked up in the text, an odd vocabulary in 16 bits
        dict(name="verify greedy 32", kind="verify", B=32, n=5, V=150001, dtype="bf16", draft=False, greedy=True),
        # one prompt continued in four ways, and its continuations returned
        dict(name="fork 4 samples", kind="fork", roots=1, forks=4, Hkv=8, D=128, P=64, dtype="bf16", lo=1000, hi=1000, pages=200),
        # sixteen prompts continued in fifteen ways each
        dict(name="fork 16 x 15", kind="fork", roots=16, forks=15, Hkv=8, D=128, P=64, dtype="bf16", lo=4000, hi=8000, pages=3000),
        # a pool half in use, its pages moved to the front
        dict(name="compact 4096", kind="compact", R=64, Hkv=8, D=128, P=64, dtype="bf16", lo=300, hi=6000, pages=4096),
        # one long instruction before 64 short chats
        dict(name="shared decode 64", kind="shared", groups=1, each=64, alone=0, Hq=32, Hkv=8, D=128, P=64, dtype="bf16", plo=8192, phi=8192,
             lo=16, hi=600, q=1, window=0, lse=False),
        # eight instructions of several lengths, sixteen chats each, and some without one
        dict(name="shared groups 8 x 16", kind="shared", groups=8, each=16, alone=5, Hq=64, Hkv=8, D=128, P=32, dtype="f16", plo=1000, phi=6000,
             lo=100, hi=2000, q=1, window=0, lse=True),
        # two documents, eight requests each that draft; one kv head of 256, the last tokens of a window
        dict(name="shared drafts window", kind="shared", groups=2, each=8, alone=0, Hq=16, Hkv=1, D=256, P=64, dtype="bf16", plo=20000, phi=30000,
             lo=10, hi=700, q=5, window=16384, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["rope", "verify", "fork", "compact", "shared", "shared"])
    P, D, dtype = rng.choice([32, 64, 96, 128, 256]), rng.choice([64, 128, 256]), rng.choice(["bf16", "f16"])
    Hkv, G = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
    if kind == "rope":
        D, T = rng.choice([48, 64, 80, 96, 128, 192, 256]), _log(rng, 1, 16384)
        H = min(G * Hkv, max(Hkv, 16384 * 32 * 128 // (T * D) // Hkv * Hkv))
        return dict(kind=kind, T=T, Hq=H, Hkv=Hkv, D=D, R=D if rng.random() < 0.5 else 2 * rng.randrange(1, D // 2 + 1),
                    dtype=rng.choice(["bf16", "f16", "f32"]) if T < 8000 else dtype, interleaved=rng.random() < 0.4,
                    inverse=rng.random() < 0.3, far=_log(rng, 100, 1 << 20), stretch=rng.choice([1.0, 1.0, 4.0, 40.0]))
    if kind == "verify":
        V, n = _log(rng, 500, 160000), rng.randrange(1, 10)
        B = _log(rng, 1, max(2, min(256, 49_000_000 // (V * n))))
        return dict(kind=kind, B=B, n=n, V=V, dtype=rng.choice(["f32", "f32", "bf16", "f16"]), draft=rng.random() < 0.6, greedy=rng.random() < 0.3)
    if kind == "fork":
        roots, hi = _log(rng, 1, 24), _log(rng, 10, 8000)
        forks = _log(rng, 1, max(2, 240 // roots))
        lo = max(1, hi // rng.choice([1, 2, 7]))
        return dict(kind=kind, roots=roots, forks=forks, Hkv=Hkv, D=min(D, 128), P=P, dtype=dtype, lo=lo, hi=hi,
                    pages=roots * (hi // P + 2) + roots * forks + rng.randrange(1, 50))
    if kind == "compact":
        R, hi = _log(rng, 1, 200), _log(rng, 20, 8000)
        hi = min(hi, 200000 // R)
        return dict(kind=kind, R=R, Hkv=Hkv, D=min(D, 128), P=P, dtype=dtype, lo=max(1, hi // rng.choice([1, 5, 20])), hi=hi,
                    pages=int((R * (hi // P + 1) + 1) * rng.choice([1.0, 1.3, 2.0])))
    phi, q = _log(rng, 40, 30000), rng.choice([1, 1, 1, 2, 4, 7])
    groups, hi = _log(rng, 1, 12), _log(rng, 5, 3000)
    each = max(1, min(_log(rng, 1, 64), 600_000 // (groups * (phi + hi))))
    while groups * each * (phi + hi) * Hkv * D > 1_300_000_000:
        phi, each = max(20, phi * 2 // 3), max(1, each * 2 // 3)
    return dict(kind=kind, groups=groups, each=each, alone=rng.choice([0, 0, 1, 3]), Hq=G * Hkv, Hkv=Hkv, D=D, P=P, dtype=dtype,
                plo=max(1, phi // rng.choice([1, 3])), phi=phi, lo=max(1, hi // rng.choice([1, 4, 30])), hi=hi, q=q,
                window=rng.choice([0, 0, 0, _log(rng, 16, 20000)]), lse=rng.random() < 0.5)


def _of(case):
    """Random numbers of the case alone, so that work() can count lengths."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lens(case):
    r = _of(case)
    if case["kind"] == "verify":
        n = [r.randrange(1, case["n"] + 1) for _ in range(case["B"])]
        n[0] = case["n"]
        if case["B"] > 8:
            n[case["B"] // 2] = 0                 # a slot of the batch that no request holds
        return n
    if case["kind"] in ("fork", "compact"):
        return [_log(r, case["lo"], case["hi"]) for _ in range(case["roots"] if case["kind"] == "fork" else case["R"])]
    # prefix of each group (whole pages are shared), tokens of each request behind it
    prefix = [_log(r, case["plo"], case["phi"]) for _ in range(case["groups"])]
    tails = [_log(r, case["lo"], case["hi"]) for _ in range(case["groups"] * case["each"] + case["alone"])]
    return prefix, [max(t, case["q"]) for t in tails]


def _page_bytes(case, tokens):
    return case["Hkv"] * 2 * (-(-tokens // 32) * 16 * case["D"] + 2 * tokens)


def work(case):
    kind = case["kind"]
    if kind == "rope":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2) + 4 * case["T"],
                "flops": 3 * case["T"] * (case["Hq"] + case["Hkv"]) * case["R"]}
    if kind == "verify":
        n, size = _lens(case), 4 if case["dtype"] == "f32" else 2
        if case["greedy"]:
            return {"bytes": sum(n) * case["V"] * size, "flops": 0}
        return {"bytes": sum(x > 0 for x in n) * case["V"] * size * (2 if case["draft"] else 1) + 12 * sum(n), "flops": 0}
    if kind == "fork":
        lens, F, P = _lens(case), case["forks"], case["P"]
        tails = sum(F * 2 * _page_bytes(case, n % P) for n in lens)
        # entries read and written by the fork, read and cleared by the return; shares read and written twice
        return {"bytes": tails + sum(F * 16 * (-(-n // P)) + 16 * (n // P) for n in lens), "flops": 0}
    if kind == "compact":
        held = [-(-n // case["P"]) for n in _lens(case)]
        used = sum(held)
        moved = used * max(0, case["pages"] - used) // case["pages"]
        return {"bytes": moved * 2 * _page_bytes(case, case["P"]) + 8 * used + 12 * case["pages"], "flops": 0}
    prefix, tails = _lens(case)
    q, D, keys, pairs = case["q"], case["D"], 0, 0
    for b, t in enumerate(tails):
        g = b // case["each"]
        p = prefix[g] // case["P"] * case["P"] if g < case["groups"] else 0
        pos = np.arange(p + t - q, p + t)
        lo = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros(q, int)
        pairs += int((pos + 1 - lo).sum())
        keys += p + t - max(p, int(lo[0]))
        if g < case["groups"] and b % case["each"] == 0:
            keys += max(0, p - int(lo[0]))
    rows = q * len(tails) * case["Hq"]
    return {"bytes": keys * case["Hkv"] * (D + 4) + rows * D * 4 + (4 * rows if case["lse"] else 0), "flops": 4 * D * case["Hq"] * pairs}


# ---- inputs ------------------------------------------------------------------

def _codebook(H, g):
    """Sorted levels such as k-means gives for rows scaled to a largest magnitude of one."""
    u = torch.linspace(-1, 1, 16, device=DEV) * 0.97
    c = u.sign() * u.abs() ** 1.25 + 0.02 * torch.randn(2, H, 16, device=DEV, generator=g)
    return c.clamp(-1, 1).sort(-1).values.half()


def _cache(pages, H, D, P, dtype, g):
    """A cache in use: codes as frequent as those of normal values, scales of rows of many magnitudes."""
    edges = torch.linspace(-2.6, 2.6, 15, device=DEV)
    cdf = 0.5 * (1 + torch.erf(edges / math.sqrt(2)))
    nib = torch.searchsorted(cdf, (torch.arange(256, device=DEV) + 0.5) / 256).to(torch.uint8)
    n = pages * H * 2 * (P // 32) * 16 * D
    codes = torch.empty(n, dtype=torch.uint8, device=DEV)
    for at in range(0, n, 1 << 27):
        m = min(1 << 27, n - at)
        a = torch.randint(0, 256, (2, m), device=DEV, generator=g, dtype=torch.int32)
        codes[at:at + m] = nib[a[0]] | nib[a[1]] << 4
    scales = 2.7 * torch.exp(0.3 * torch.randn(pages, H, 2, P, device=DEV, generator=g))
    return codes.view(pages, H, 2, P // 32, 16 * D), scales.to(dtype)


BASE, SLOW, FAST, TRAINED = 10000.0, 1.0, 32.0, 4096


def _frequencies(case):
    """Radians a position of each pair: BASE^(-2 i / R).  A stretched context
    divides the slow ones by the stretch, leaves those that turn FAST times or
    more over the trained length, and goes from one to the other in between."""
    f = BASE ** (-torch.arange(0, case["R"], 2, dtype=torch.float64, device=DEV) / case["R"])
    s = case["stretch"]
    keep = ((TRAINED * f / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0, 1)
    return keep * f + (1 - keep) * f / s, 1 + 0.1 * math.log(s)


def _rope_state(case, g):
    T, Hq, H, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    dt = TYPES[case["dtype"]]
    qkv = torch.randn(T, (Hq + 2 * H) * D, device=DEV, generator=g).to(dt)
    # runs of consecutive positions from anywhere in the contexts; one token in 50 is padding
    run = max(1, T // 7)
    start = torch.randint(0, case["far"], (T // run + 1,), device=DEV, generator=g)
    i = torch.arange(T, device=DEV)
    pos = start[i // run] + i % run
    pos[torch.rand(T, device=DEV, generator=g) < 0.02] = -1
    f, factor = _frequencies(case)
    st = dict(q=qkv[:, :Hq * D].unflatten(1, (Hq, D)), k=qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D)), pos=pos.int(),
              qo=torch.empty(T, Hq, D, dtype=dt, device=DEV), ko=torch.empty(T, H, D, dtype=dt, device=DEV), f=f, factor=factor)
    if own:
        import exact_lloyd_means_amd as fk
        st["turns"] = fk.rope_turns(case["R"], BASE, stretch=case["stretch"], trained=TRAINED, slow=SLOW, fast=FAST, device=DEV)
    return st


def _verify_state(case, g):
    n, V, dt = _lens(case), case["V"], TYPES[case["dtype"]]
    n = [n[i] for i in torch.randperm(case["B"], device=DEV, generator=g).tolist()]
    T = sum(n)
    logits = 2.5 * torch.randn(T, V, device=DEV, generator=g)
    near = logits + 0.6 * torch.randn(T, V, device=DEV, generator=g)
    p, q = (torch.softmax(x, -1).to(dt) for x in (logits, near))
    # drafts drawn from the small model (by a race of exponentials), or for greedy decoding its most likely ones
    race = near if case["greedy"] else near - torch.log(-torch.log(torch.rand(T, V, device=DEV, generator=g).clamp(1e-9, 1 - 1e-7)))
    drafts = race.argmax(-1)
    tokens = torch.roll(drafts, 1)
    u = torch.rand(T, device=DEV, generator=g)
    pick = torch.rand(case["B"], device=DEV, generator=g)
    seq = torch.randint(0, 5000, (case["B"],), device=DEV, generator=g) + torch.tensor(n, device=DEV)
    st = dict(cu=torch.tensor([0] + list(np.cumsum(n)), **I32), tokens=tokens.int(), p=p, q=q if case["draft"] else None,
              u=None if case["greedy"] else u, pick=None if case["greedy"] else pick, seq=seq.int(),
              accepted=torch.empty(case["B"], **I32), emitted=torch.empty(T, **I32), keep=torch.empty(case["B"], **I32))
    if own:
        import exact_lloyd_means_amd as fk
        st["ws"] = fk.verify_workspace(st["cu"], st["p"])
    return st


def _pool(case, lens, rows, g):
    """A block table whose first rows hold these lengths in pages taken in any order, the free list and the shares."""
    P, N = case["P"], case["pages"]
    held = torch.tensor([-(-n // P) for n in lens] + [0] * (rows - len(lens)), device=DEV)
    M = case["hi"] // P + 1
    used = torch.arange(M, device=DEV) < held[:, None]
    total = sum(-(-n // P) for n in lens)
    ids = torch.randperm(N, device=DEV, generator=g).int()
    table = torch.full((rows, M), -1, **I32)
    table[used] = ids[:total]
    free = torch.full((N,), -1, **I32)
    free[:N - total] = ids[total:]
    return dict(table=table, lens=torch.tensor(list(lens) + [0] * (rows - len(lens)), **I32), free=free, P=P,
                count=torch.tensor([N - total], **I32), shares=torch.zeros(N, **I32))


def _fork_state(case, seed, g):
    F, lens = case["forks"], _lens(case)
    n = case["roots"]
    lens = [lens[i] for i in random.Random(seed).sample(range(n), n)]
    st = _pool(case, lens, n * (1 + F), g)
    st["rows"] = torch.arange(n, n * (1 + F), **I32)
    st["src"] = torch.arange(n, **I32).repeat_interleave(F)
    st["all"], st["none"] = torch.full((n * F,), 2 ** 31 - 1, **I32), torch.zeros(n * F, **I32)
    st["copies"], st["back"] = (torch.empty(n * F, 3, **I32) for _ in range(2))
    st["codes"], st["scales"] = _cache(case["pages"], case["Hkv"], case["D"], case["P"], TYPES[case["dtype"]], g)
    if own:
        import exact_lloyd_means_amd as fk
        st["ws"] = fk.kv_fork_workspace(n * F, st["table"], st["shares"])
    return st


def _compact_state(case, seed, g):
    lens = _lens(case)
    lens = [lens[i] for i in random.Random(seed).sample(range(case["R"]), case["R"])]
    st = _pool(case, lens, case["R"], g)
    N = case["pages"]
    st |= dict(new_table=torch.empty_like(st["table"]), new_free=torch.full((N,), -1, **I32), left=torch.empty(1, **I32),
               new_shares=torch.empty(N, **I32), moves=torch.empty((N + 1) // 2, 3, **I32))
    st["codes"], st["scales"] = _cache(N, case["Hkv"], case["D"], case["P"], TYPES[case["dtype"]], g)
    if own:
        import exact_lloyd_means_amd as fk
        st["ws"] = fk.kv_compact_workspace(st["shares"])
    return st


def _shared_state(case, g):
    P, D, H, dt, each = case["P"], case["D"], case["Hkv"], TYPES[case["dtype"]], case["each"]
    prefix, tails = _lens(case)
    prefix = [p // P * P for p in prefix]
    B, q = len(tails), case["q"]
    of = [b // each if b // each < len(prefix) else -1 for b in range(B)]
    seq = [t + (prefix[o] if o >= 0 else 0) for t, o in zip(tails, of)]
    M = max(1, max(-(-s // P) for s in seq))
    need = sum(prefix) // P + sum(-(-t // P) for t in tails)
    ids = torch.randperm(need + 3, device=DEV, generator=g).int().cpu().numpy()
    table, at, first = np.full((B, M), -1, np.int32), sum(prefix) // P, np.cumsum([0] + prefix) // P
    for b, (t, o) in enumerate(zip(tails, of)):
        n, more = prefix[o] // P if o >= 0 else 0, -(-t // P)
        table[b, :n] = ids[first[o]:first[o] + n] if n else []
        table[b, n:n + more] = ids[at:at + more]
        at += more
    st = dict(table=torch.from_numpy(table).to(DEV), seq=torch.tensor(seq, **I32), Q=q, S=max(seq),
              cu=torch.arange(0, q * B + 1, q, **I32), cug=torch.arange(0, each * len(prefix) + 1, each, **I32),
              prefix=torch.tensor(prefix, **I32), cb=_codebook(H, g), scale=1 / math.sqrt(D),
              q=(2 * torch.randn(q * B, case["Hq"], D, device=DEV, generator=g)).to(dt),
              out=torch.empty(q * B, case["Hq"], D, dtype=dt, device=DEV), lse=torch.empty(q * B, case["Hq"], device=DEV) if case["lse"] else None)
    st["codes"], st["scales"] = _cache(need + 3, H, D, P, dt, g)
    if own:
        import exact_lloyd_means_amd as fk
        st["ws"] = fk.kv4_attention_shared_workspace(st["q"], st["seq"], st["prefix"], st["codes"], q)
    return st


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    kind = case["kind"]
    st = (_rope_state(case, g) if kind == "rope" else _verify_state(case, g) if kind == "verify" else _fork_state(case, seed, g)
          if kind == "fork" else _compact_state(case, seed, g) if kind == "compact" else _shared_state(case, g))
    return st | {"case": case, "kind": kind}


# ---- the operators in plain form -----------------------------------------------

def _rotate(x, c, s, R, interleaved):
    y = x.float()
    a, b = (y[..., :R:2], y[..., 1:R:2]) if interleaved else (y[..., :R // 2], y[..., R // 2:R])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, y[..., R:]), -1)


def _rope(st):
    case = st["case"]
    angle = st["pos"].double()[:, None] * st["f"]
    c, s = (angle.cos() * st["factor"]).float()[:, None], (angle.sin() * st["factor"]).float()[:, None]
    s = -s if case["inverse"] else s
    there = (st["pos"] >= 0)[:, None, None]
    q, k = (torch.where(there, _rotate(x, c, s, case["R"], case["interleaved"]).to(x.dtype), x) for x in (st["q"], st["k"]))
    return {"q": q, "k": k}


def _weights(x):
    """Values in 0 .. 1 as whole multiples of 2^-42, so that sums of them do not round."""
    return (torch.where(x > 0, x, 0).clamp(max=1) * 2.0 ** 42).long()


def _verify(st):
    cu, tokens, p, q = st["cu"].long(), st["tokens"].long(), st["p"], st["q"]
    T, V = p.shape
    B = cu.numel() - 1
    r = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:], r, right=True)
    last = r + 1 == cu[b + 1]
    d = tokens.roll(-1)
    good = ~last & (d >= 0) & (d < V)
    at = d.clamp(0, V - 1)[:, None]
    if st["u"] is None:
        x = p.float()
        x = torch.where(x == x, x, -math.inf)
        best = torch.where(x == x.amax(-1, keepdim=True), torch.arange(V, device=DEV), V).amin(-1)
        good &= best == d
    else:
        chance = st["u"].double() * (1 if q is None else q.gather(1, at)[:, 0].double())
        good &= chance < p.gather(1, at)[:, 0].double()
    stop = torch.full((B,), T, device=DEV).scatter_reduce_(0, b, torch.where(good, T, r), "amin")     # row of the first draft refused, or the last
    row = stop.clamp(max=T - 1)
    some = cu[1:] > cu[:-1]
    accepted = torch.where(some, stop - cu[:-1], 0)
    if st["u"] is None:
        token = best[row]
    else:
        x, refused = p[row].float(), ~last[row][:, None]
        away = (torch.arange(V, device=DEV) == at[row]).float() * 2 if q is None else q[row].float()
        w, plain = _weights(torch.where(refused, x - away, x)), _weights(x)
        w = torch.where(w.sum(-1, keepdim=True) > 0, w, plain)
        upto = w.cumsum(-1)
        total = upto[:, -1]
        s = (st["pick"].double() * 2.0 ** 31).long().clamp(0, 2 ** 31 - 1)
        point = 2 * (total >> 32) * s + ((total & 0xffffffff) * s >> 31)
        token = torch.where(total > 0, torch.searchsorted(upto, point[:, None], right=True)[:, 0], -1)
    i = r - cu[b]
    emitted = torch.where(i < accepted[b], d, torch.where(i == accepted[b], token[b], -1))
    keep = st["seq"].long() - torch.where(some, cu[1:] - cu[:-1] - 1 - accepted, 0)
    return {"accepted": accepted.int(), "emitted": emitted.int(), "keep": keep.int()}


def _fork(st, rows, src, keep):
    """Rows of the table become the first `keep` tokens of other rows, all at once; src None: of themselves.  Returns what is to be copied."""
    table, lens, shares, free, count, P = st["table"], st["lens"], st["shares"], st["free"], st["count"], st["P"]
    (R, M), N, n = table.shape, shares.numel(), rows.numel()
    i = torch.arange(n, device=DEV)
    page = torch.arange(M, device=DEV)
    r = torch.where((rows >= 0) & (rows < R), rows, R).long()
    s = r if src is None else torch.where((src >= 0) & (src < R), src, R).long()
    length = torch.cat((lens, lens.new_zeros(1))).long()
    least = torch.full((R + 1,), 2 ** 31 - 1, device=DEV).scatter_reduce_(0, r, keep.long(), "amin")[r]
    L = least.clamp(min=0).minimum(length[s])
    turn = torch.full((R + 1,), n, device=DEV).scatter_reduce_(0, r, i, "amin")[r]
    act = (turn == i) & (r < R) & ~((s == r) & (L == length[r]))
    rows_of = torch.cat((table, table.new_full((1, M), -1))).long()
    old, new, W, tail = rows_of[r], rows_of[s], L // P, L % P
    held = (length[r] + P - 1) // P
    mine = act[:, None] & (page < held[:, None]) & (old >= 0)
    whole = act[:, None] & (page < W[:, None]) & (new >= 0)
    end = new.gather(1, W.clamp(max=M - 1)[:, None])[:, 0]
    end = torch.where(act & (tail > 0) & (end >= 0), end, N)
    zeros = torch.zeros(N + 1, dtype=torch.int64, device=DEV)
    at = torch.where(mine, old, N).flatten()
    drop = zeros.scatter_add(0, at, torch.ones_like(at))
    to = torch.where(whole, new, N).flatten()
    base = torch.cat((shares.long() + 1, zeros[:1])) - drop + zeros.scatter_add(0, to, torch.ones_like(to))
    first = (zeros + n).scatter_reduce(0, end, i, "amin")
    moves = (end < N) & (base[end] == 0) & (first[end] == i)
    copied = (end < N) & ~moves
    refs = base + ((base == 0) & (first < n))
    entry = torch.arange(n * M, device=DEV)
    gone = (at < N) & (refs[at] == 0) & ((zeros + n * M).scatter_reduce(0, at, entry, "amin")[at] == entry)
    # pages returned go behind the list, those for the copies are its last ones
    longer = torch.cat((free, free.new_empty(1)))
    longer[torch.where(gone, count + gone.cumsum(0) - 1, N)] = at.int()
    free.copy_(longer[:N])
    have = count + gone.sum()
    got = torch.minimum(copied.sum(), have)
    rank = copied.cumsum(0) - 1
    fresh = torch.where(copied & (rank < got), free[(have - got + rank).clamp(0, N - 1)], -1)
    count.copy_(have - got)
    shares.copy_((refs[:N] - 1).clamp(min=0))
    tail_page = torch.where(moves, end, fresh)
    row = torch.where(whole, new, torch.where((page == W[:, None]) & (tail_page >= 0)[:, None], tail_page[:, None], -1))
    row = torch.where((page >= held[:, None]) & (page > W[:, None]), old, row)
    put = torch.where(act, r, R)
    rows_of[put] = row
    table.copy_(rows_of[:R])
    length[put] = torch.where(tail_page >= 0, L, W * P)
    lens.copy_(length[:R])
    none = fresh < 0
    return torch.stack((torch.where(none, -1, end), fresh, torch.where(none, 0, tail)), -1).int()


def _copy(st, list_):
    """Whole blocks of the first tokens of pages to other pages; (source, destination, tokens), negative: none."""
    codes, scales = st["codes"], st["scales"]
    src, dst, n = list_.long().unbind(-1)
    there = dst >= 0
    src, dst, n = src[there], dst[there], n[there]
    block = torch.arange(codes.shape[3], device=DEV) < ((n + 31) // 32)[:, None]
    part = block[:, None, None, :, None].expand(-1, *codes.shape[1:])
    codes[dst] = torch.where(part, codes[src], codes[dst])
    scales[dst] = torch.where(block.repeat_interleave(32, -1)[:, None, None], scales[src], scales[dst])


def _pages(st):
    """The state's own buffers; scales are moved, not computed with, so their bits are compared."""
    names = ("table", "lens", "shares", "free", "count") if st["kind"] == "fork" else ("new_table", "new_free", "left", "new_shares", "moves")
    return {k: st[k] for k in (*names, "codes")} | {"scales": st["scales"].view(torch.int16)}


def _fork_and_back(st):
    copies = _fork(st, st["rows"], st["src"], st["all"])
    _copy(st, copies)
    forked = st["table"].clone()
    return {"copies": copies, "forked": forked, "back": _fork(st, st["rows"], None, st["none"])} | _pages(st)


def _compact(st):
    table, N, P, M = st["table"], st["shares"].numel(), st["P"], st["table"].shape[1]
    ids = torch.arange(N, device=DEV)
    free = torch.zeros(N + 1, dtype=torch.int64, device=DEV)
    free[torch.where(ids < st["count"], st["free"], N).long()] = 1
    free = free[:N] > 0
    U = N - free.sum()
    hole, mover = free & (ids < U), ~free & (ids >= U)
    rank_h, rank_m = hole.cumsum(0) - 1, mover.cumsum(0) - 1
    pairs = torch.full((N + 1, 3), -1, device=DEV)
    pairs[:, 2] = 0
    pairs[torch.where(hole, rank_h, N), 1] = ids
    pairs[torch.where(mover, rank_m, N), 0] = ids
    pairs[torch.where(mover, rank_m, N), 2] = P
    to = torch.where(mover, pairs[rank_m.clamp(min=0), 1], ids)
    held = (st["lens"] + P - 1) // P
    mine = (torch.arange(M, device=DEV) < held[:, None]) & (table >= 0)
    st["new_table"].copy_(torch.where(mine, to[table.clamp(min=0).long()], table))
    shares = torch.zeros(N + 1, **I32)
    shares[torch.where(free, N, to)] = st["shares"]
    st["new_shares"].copy_(shares[:N])
    st["new_free"].copy_(torch.where(ids < N - U, N - 1 - ids, st["new_free"]))
    st["left"].copy_(N - U)
    st["moves"].copy_(pairs[:st["moves"].shape[0]])
    _copy(st, st["moves"])
    return _pages(st)


# axes of a block's bytes: k and v of a head of D, and the order that makes them (token, byte of the row)
BLOCKS = {(64, 0): ((4, 4, 4, 2, 8), (1, 3, 2, 0, 4)), (128, 0): ((2, 4, 4, 4, 16), (2, 0, 3, 1, 4)),
          (256, 0): ((2, 2, 4, 4, 4, 16), (3, 0, 4, 2, 1, 5)), (64, 1): ((4, 16, 8, 2), (0, 2, 1, 3)),
          (128, 1): ((2, 4, 16, 4, 4), (1, 0, 3, 2, 4)), (256, 1): ((2, 2, 4, 16, 4, 4), (2, 1, 4, 3, 0, 5))}


def _rows(x, D, kv):
    """(..., 16 D) bytes of blocks -> (..., 32, D/2): a token's bytes in the order of its dimensions."""
    shape, order = BLOCKS[D, kv]
    n = x.dim() - 1
    x = x.reshape(*x.shape[:-1], *shape)
    return x.permute(*range(n), *(n + i for i in order)).reshape(*x.shape[:n], 32, D // 2)


def _values(rows, scale, cb):
    """(..., H, S, D/2) bytes and (..., H, S) scales -> the float32 values (..., H, S, D); cb (H, 16)."""
    codes = torch.stack((rows & 15, rows >> 4), -1).flatten(-2).int()
    codes += 16 * torch.arange(cb.shape[0], device=DEV, dtype=torch.int32)[:, None, None]
    return cb.float().view(-1).index_select(0, codes.view(-1)).view(codes.shape) * scale.float()[..., None]


def _shared(st):
    c = st["case"]
    D, H, P, Q = c["D"], c["Hkv"], c["P"], st["Q"]
    B, M, G = *st["table"].shape, c["Hq"] // c["Hkv"]
    table = st["table"].clamp(min=0).long()
    k, v = (_values(_rows(st["codes"][:, :, kv][table], D, kv).permute(0, 2, 1, 3, 4, 5).reshape(B, H, M * P, D // 2),
                    st["scales"][:, :, kv][table].transpose(1, 2).reshape(B, H, M * P), st["cb"][kv]) for kv in (0, 1))
    q = st["q"].float().view(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    s = (q @ k.transpose(-1, -2) * st["scale"]).view(B, H, G, Q, M * P)
    pos = (st["seq"] - Q)[:, None, None] + torch.arange(Q, device=DEV)[:, None]
    j = torch.arange(M * P, device=DEV)
    seen = j <= pos
    if c["window"]:
        seen = seen & (j > pos - c["window"])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B * Q, H * G)
    o = (p / total).view(B, H, G * Q, M * P) @ v
    o = o.view(B, H, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B * Q, H * G, D)
    return {"out": o.to(st["q"].dtype), "lse": lse if c["lse"] else None}


def run(st):
    kind, c = st["kind"], st["case"]
    if not own:
        return {"rope": _rope, "verify": _verify, "fork": _fork_and_back, "compact": _compact, "shared": _shared}[kind](st)
    import exact_lloyd_means_amd as fk
    if kind == "rope":
        fk.fk_rope(st["q"], st["k"], st["pos"], st["turns"], st["qo"], st["ko"], interleaved=c["interleaved"], inverse=c["inverse"],
                   factor=st["factor"])
        return {"q": st["qo"], "k": st["ko"]}
    if kind == "verify":
        fk.fk_verify(st["cu"], st["tokens"], st["p"], st["accepted"], st["emitted"], draft=None if c["greedy"] else st["q"], accept=st["u"],
                     pick=st["pick"], seq_lens=st["seq"], keep=st["keep"], ws=st["ws"])
        return {k: st[k] for k in ("accepted", "emitted", "keep")}
    if kind == "fork":
        pool = (st["P"], st["table"], st["lens"], st["shares"], st["free"], st["count"])
        fk.fk_kv_fork(st["rows"], st["src"], st["all"], *pool, st["copies"], ws=st["ws"])
        fk.fk_kv4_copy(st["copies"], st["codes"], st["scales"])
        forked = st["table"].clone()
        fk.fk_kv_fork(st["rows"], None, st["none"], *pool, st["back"], ws=st["ws"])
        return {"copies": st["copies"], "forked": forked, "back": st["back"]} | _pages(st)
    if kind == "compact":
        fk.fk_kv_compact(st["P"], st["table"], st["lens"], st["shares"], st["free"], st["count"], st["new_table"], st["new_shares"],
                         st["new_free"], st["left"], st["moves"], ws=st["ws"])
        fk.fk_kv4_copy(st["moves"], st["codes"], st["scales"])
        return _pages(st)
    fk.fk_kv4_attention_shared(st["q"], st["cu"], st["seq"], st["table"], st["cug"], st["prefix"], st["cb"], st["codes"], st["scales"],
                               st["out"], st["Q"], scale=st["scale"], window=c["window"], lse=st["lse"], ws=st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


# ---- the definitions in 64 bits ---------------------------------------------------

def _address(D, kv):
    """Byte and shift of the code of (token t of a block, dimension d), from the layout's definition."""
    t, d = np.meshgrid(np.arange(32), np.arange(D), indexing="ij")
    if kv == 0:                                     # a lane (16 g + m) holds D/4 dimensions of two tokens
        lane, at = 16 * (d // (D // 4)) + 4 * (t // 8) + t % 4, t // 4 % 2 * (D // 8) + d % (D // 4) // 2
    else:                                           # a lane (16 g + r) holds D/16 dimensions of eight tokens
        w = d % (D // 16)
        lane, at = 16 * (t // 8) + d // (D // 16), (w // 8) * 32 + t % 8 * min(4, D // 32) + w % 8 // 2
    return torch.from_numpy(at // 16 * 1024 + lane * 16 + at % 16).to(DEV), torch.from_numpy(d % 2 * 4).to(DEV)


def _exact_rope(case, st):
    """Pairs as complex numbers: z exp(i angle) factor."""
    R, pos, got = case["R"], st["pos"].tolist(), {}
    pair = np.arange(R // 2)
    f = BASE ** (-2.0 * pair / R)
    turns = TRAINED * f / (2 * np.pi)
    share = np.minimum(1, np.maximum(0, (turns - SLOW) / (FAST - SLOW)))
    f = f / case["stretch"] * (1 - share) + f * share
    angle = np.array(pos, dtype=np.float64)[:, None] * f * (-1 if case["inverse"] else 1)
    z = torch.from_numpy(np.exp(1j * angle) * (0.1 * math.log(case["stretch"]) + 1)).to(DEV)[:, None]
    a, b = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + R // 2)
    for name in ("q", "k"):
        x = st[name].double()
        y = x.clone()
        w = torch.complex(x[..., a], x[..., b]) * z
        y[..., a], y[..., b] = w.real, w.imag
        got[name] = torch.where((st["pos"] < 0)[:, None, None], x, y)
    return got


def exact(case, seed):
    if case["kind"] not in ("rope", "shared") or work(case)["flops"] > 3e12:
        return None
    st = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_rope(case, st)
    D, P, H, n = case["D"], case["P"], case["Hkv"], st["Q"]
    G, cb = case["Hq"] // H, st["cb"].double()
    place = [_address(D, kv) for kv in (0, 1)]
    out, lse = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV), torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=DEV)
    for b, S in enumerate(st["seq"].tolist()):
        q = st["q"][b * n:(b + 1) * n].double().view(n, H, G, D)
        first = max(0, S - n - case["window"]) if case["window"] else 0
        j = torch.arange(first, S, device=DEV)
        page, t = st["table"][b].long()[j // P], j % P
        pos = torch.arange(S - n, S, device=DEV)[:, None]
        seen = (j <= pos) & (j > pos - (case["window"] or S + 1))
        for h in range(H):
            k, v = (cb[w, h][(torch.gather(st["codes"][page, h, w, t // 32], 1, place[w][0][t % 32]).int() >> place[w][1][t % 32] & 15).long()]
                    * st["scales"][page, h, w, t].double()[:, None] for w in (0, 1))
            s = (q[:, h].reshape(-1, D) @ k.T * st["scale"]).view(n, G, len(j)).masked_fill(~seen[:, None], -math.inf)
            l = torch.logsumexp(s, -1)
            lse[b * n:(b + 1) * n].view(n, H, G)[:, h] = l
            out[b * n:(b + 1) * n].view(n, H, G, D)[:, h] = (torch.exp(s - l[..., None]).view(-1, len(j)) @ v).view(n, G, D)
    return {"out": out, "lse": lse if case["lse"] else None}
