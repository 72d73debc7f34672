"""Operators of the paged 4-bit cache, as they are measured: the page plan of
a serving step (block tables and slot maps from request lengths), rows
appended to the cache and read back, and attention over it.

A cache row is one token's k or v of one kv head: D codes of 4 bits, indices
into the head's 16 sorted codebook values, and one scale, the row's largest
magnitude in the cache's 16-bit type.  The row stands for codebook[code] * scale.

Storage:  codes     uint8 (pages, kv heads, 2, page/32, 16 D): k then v, blocks of 32 tokens
          scales    (pages, kv heads, 2, page) in the cache's type
          codebook  float16 (2, kv heads, 16)
"""
import math
import random

import numpy as np
import torch

own = False                               # whether run() makes the package's calls; it is imported only there

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small server: 64 requests, one new token each
        dict(name="plan decode 64", kind="plan", B=64, P=64, pages=128, ctx=2000, new=1, cap=64),
        # a large step: thousands of requests that decode beside prompts that arrive
        dict(name="plan mixed 3000", kind="plan", B=3000, P=32, pages=512, ctx=3000, new=700, cap=1 << 20),
        # the new tokens of one decode step, slices of the fused qkv projection
        dict(name="append decode 64", kind="append", T=64, Hq=32, Hkv=8, D=128, P=64, dtype="bf16", run=1),
        # a prompt's tokens at once
        dict(name="append prompt 16384", kind="append", T=16384, Hq=32, Hkv=8, D=128, P=64, dtype="bf16", run=4096),
        # odd lengths, three kv heads, small heads, fp16
        dict(name="append ragged 5001", kind="append", T=5001, Hq=6, Hkv=3, D=64, P=32, dtype="f16", run=333),
        # one chat at its start: the smallest call
        dict(name="attend one", kind="attend", B=1, Hq=32, Hkv=8, D=128, P=64, dtype="bf16", lo=257, hi=257, q=1,
             causal=True, window=0, lse=False),
        # an ordinary decode batch of ragged contexts
        dict(name="attend decode 64", kind="attend", B=64, Hq=32, Hkv=8, D=128, P=64, dtype="bf16", lo=512, hi=8192, q=1,
             causal=True, window=0, lse=False),
        # many short chats, eight query heads to a kv head
        dict(name="attend short 256", kind="attend", B=256, Hq=64, Hkv=8, D=128, P=32, dtype="f16", lo=16, hi=600, q=1,
             causal=True, window=0, lse=False),
        # a few very long documents
        dict(name="attend long 3", kind="attend", B=3, Hq=32, Hkv=8, D=128, P=128, dtype="bf16", lo=66000, hi=131072, q=1,
             causal=True, window=0, lse=True),
        # draft tokens verified together (q per request), a window, one kv head of 256
        dict(name="attend verify window", kind="attend", B=16, Hq=16, Hkv=1, D=256, P=64, dtype="bf16", lo=900, hi=20000, q=5,
             causal=True, window=4096, lse=True),
        # ragged prompts from their first token
        dict(name="attend prompt 6", kind="attend", B=6, Hq=32, Hkv=8, D=128, P=64, dtype="bf16", lo=1000, hi=4096, q=4096,
             causal=True, window=0, lse=False),
        # a chunk of a prompt behind a long context, heads of 64
        dict(name="attend chunk 2", kind="attend", B=2, Hq=24, Hkv=8, D=64, P=64, dtype="f16", lo=12000, hi=20000, q=512,
             causal=True, window=0, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["plan", "append", "append", "attend", "attend", "attend"])
    P = rng.choice([32, 64, 96, 128, 256])
    if kind == "plan":
        B, new = _log(rng, 1, 4000), rng.choice([1, 1, _log(rng, 2, 2000)])
        return dict(kind=kind, B=B, P=P, pages=_log(rng, 40, 600), ctx=_log(rng, 30, 8000), new=new,
                    cap=min(1 << 20, max(B, B * new // 3)))
    Hkv, D, dtype = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128, 256]), rng.choice(["bf16", "f16"])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
    if kind == "append":
        T = _log(rng, 1, 16384)
        return dict(kind=kind, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, P=P, dtype=dtype, run=_log(rng, 1, max(2, T)))
    base = dict(kind=kind, Hq=G * Hkv, Hkv=Hkv, D=D, P=P, dtype=dtype, causal=rng.random() < 0.8,
                window=rng.choice([0, 0, _log(rng, 16, 3000)]), lse=rng.random() < 0.5)
    if rng.random() < 0.6:          # few query rows over a long cache
        hi = _log(rng, 20, 60000)
        B = min(_log(rng, 1, 256), max(1, 250000 // hi))
        return dict(base, B=B, lo=max(1, hi // rng.choice([1, 3, 12])), hi=hi, q=rng.choice([1, 1, 1, 2, 4, 9]))
    q = _log(rng, 10, 2500)         # prompts and chunks
    hi = max(q, _log(rng, 10, 16000))
    B = max(1, min(_log(rng, 1, 16), 400_000_000 // (q * hi * G * Hkv)))
    if q * hi * G * Hkv * D > 40_000_000_000:
        hi = max(q // 2, 40_000_000_000 // (q * G * Hkv * D))
    return dict(base, B=B, lo=max(1, hi // rng.choice([1, 4])), hi=hi, q=min(q, hi))


def _lens(case):
    """(context, new) lengths of every request: of the case alone, so work() can count them."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B = case["B"]
    if case["kind"] == "plan":
        ctx = [r.randrange(0, min(2 * case["ctx"], case["pages"] * case["P"] - 1)) for _ in range(B)]
        # one request in eight brings a prompt (fresh or another turn), one in sixteen is idle, the others decode
        new = [1 if case["new"] == 1 else r.randrange(1, 2 * case["new"]) if r.random() < 0.125 else 1 for _ in range(B)]
        new = [0 if B > 8 and r.random() < 1 / 16 else n for n in new]
        return ctx, new
    seq = [_log(r, case["lo"], case["hi"]) for _ in range(B)]
    seq[0] = case["hi"]
    q = [min(case["q"], s) if case["q"] > 16 else case["q"] for s in seq]   # a few draft tokens can exceed a fresh context
    if B > 8:
        seq[B // 2] = 0                   # a slot of the batch that no request holds
    return seq, q


def work(case):
    if case["kind"] == "plan":
        ctx, new = _lens(case)
        need = sum(max(0, min(-(-(c + n) // case["P"]), case["pages"]) - -(-c // case["P"])) for c, n in zip(ctx, new))
        return {"bytes": 8 * case["B"] + 4 * case["B"] + 8 * need + 8 * case["B"] + 8 * case["cap"], "flops": 0}
    if case["kind"] == "append":
        n, D = case["T"] * case["Hkv"], case["D"]
        return {"bytes": 2 * n * D * 2 + 4 * case["T"] + n * (D + 4) + 2 * n * D * 2, "flops": 0}
    seq, q = _lens(case)
    keys, pairs = 0, 0
    for s, n in zip(seq, q):
        pos = np.arange(s - n, s)
        hi = np.minimum(pos + 1, s) if case["causal"] else np.full(n, s)
        lo = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros(n, int)
        pairs += int(np.maximum(0, np.maximum(hi, 0) - lo).sum())
        keys += max(0, int(hi.max()) - int(lo.min()))
    rows = sum(q) * case["Hq"]
    return {"bytes": keys * case["Hkv"] * (case["D"] + 4) + rows * case["D"] * 4 + (4 * rows if case["lse"] else 0),
            "flops": 4 * case["D"] * case["Hq"] * pairs}


# ---- inputs ------------------------------------------------------------------

def _codebook(H, g):
    """Sorted levels such as k-means gives for rows scaled to a largest magnitude of one: denser near zero, not symmetric."""
    u = torch.linspace(-1, 1, 16, device=DEV) * 0.97
    c = u.sign() * u.abs() ** 1.25 + 0.02 * torch.randn(2, H, 16, device=DEV, generator=g)
    return c.clamp(-1, 1).sort(-1).values.half()


def _cache(pages, H, D, P, dtype, cb, g):
    """A cache in use: codes as frequent as those of normal values, scales of rows of many magnitudes."""
    edges = torch.linspace(-2.6, 2.6, 15, device=DEV)
    cdf = 0.5 * (1 + torch.erf(edges / math.sqrt(2)))
    u = (torch.arange(256, device=DEV) + 0.5) / 256
    nib = torch.searchsorted(cdf, u).to(torch.uint8)
    n = pages * H * 2 * (P // 32) * 16 * D
    codes = torch.empty(n, dtype=torch.uint8, device=DEV)
    for at in range(0, n, 1 << 27):
        m = min(1 << 27, n - at)
        a = torch.randint(0, 256, (2, m), device=DEV, generator=g, dtype=torch.int32)
        codes[at:at + m] = nib[a[0]] | nib[a[1]] << 4
    scales = 2.7 * torch.exp(0.3 * torch.randn(pages, H, 2, P, device=DEV, generator=g))
    return codes.view(pages, H, 2, P // 32, 16 * D), scales.to(dtype)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    st = {"case": case, "kind": case["kind"]}
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["kind"] == "plan":
        ctx, new = _lens(case)
        order = random.Random(seed).sample(range(case["B"]), case["B"])
        ctx, new = [ctx[i] for i in order], [new[i] for i in order]
        B, P, M, cap = case["B"], case["P"], case["pages"], case["cap"]
        st |= dict(P=P, ctx=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32))
        held = (st["ctx"] + P - 1) // P
        total = int(held.sum()) + sum(-(-n // P) + 1 for n in new)
        ids = torch.randperm(total, device=DEV, generator=g).int()
        used = torch.arange(M, device=DEV) < held[:, None]
        st["table"] = torch.full((B, M), -1, **i32)
        st["table"][used] = ids[:int(used.sum())]
        st["free"] = ids[int(used.sum()):].contiguous()
        st["count"] = torch.tensor([st["free"].numel()], **i32)
        st |= dict(seq=torch.empty(B, **i32), cu=torch.empty(B + 1, **i32), slots=torch.empty(cap, **i32),
                   pos=torch.empty(cap, **i32), left=torch.empty(1, **i32), status=torch.empty(4, **i32))
        if own:
            import exact_lloyd_means_amd as fk
            st["ws"] = fk.kv_plan_workspace(B, DEV)
        return st
    dt, H, D, P = TYPES[case["dtype"]], case["Hkv"], case["D"], case["P"]
    st["cb"] = _codebook(H, g)
    if case["kind"] == "append":
        T, Hq = case["T"], case["Hq"]
        qkv = torch.randn(T, Hq + 2 * H, D, device=DEV, generator=g)
        qkv[:, Hq:Hq + H] *= torch.exp(0.5 * torch.randn(H, D, device=DEV, generator=g))     # channels of k that stand out
        qkv[T // 2, Hq:] = 0                                                                  # an empty row
        qkv = qkv.to(dt).view(T, -1)
        st["k"] = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        st["v"] = qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
        # runs of consecutive positions in pages taken in any order; a run's first page is partly filled; one token in 50 is padding
        run, r = case["run"], random.Random(seed)
        pages, at = [], []
        while len(at) < T:
            p = r.randrange(P)
            for _ in range(min(run, T - len(at))):
                if p % P == 0 or not pages or p < 0:
                    pages.append(len(pages))
                at.append((len(pages) - 1) * P + p % P)
                p += 1
            pages.append(len(pages))
        n = len(pages) + 1
        perm = torch.randperm(n, device=DEV, generator=g)
        slots = torch.tensor(at, device=DEV)
        slots = perm[slots // P] * P + slots % P
        slots[torch.rand(T, device=DEV, generator=g) < 0.02] = -1
        st["slots"] = slots.int()
        st["codes"], st["scales"] = _cache(n, H, D, P, dt, st["cb"], g)
        st["ko"], st["vo"] = (torch.empty(T, H, D, dtype=dt, device=DEV) for _ in range(2))
        return st
    seq, q = _lens(case)
    order = random.Random(seed).sample(range(case["B"]), case["B"])
    seq, q = [seq[i] for i in order], [q[i] for i in order]
    held = [-(-s // P) for s in seq]
    M, pages = max(1, max(held)), sum(held) + 3
    ids = torch.randperm(pages, device=DEV, generator=g).int()
    table = torch.full((case["B"], M), -1, **i32)
    table[torch.arange(M, device=DEV) < torch.tensor(held, device=DEV)[:, None]] = ids[:sum(held)]
    T = sum(q)
    st["codes"], st["scales"] = _cache(pages, H, D, P, dt, st["cb"], g)
    st |= dict(table=table, seq=torch.tensor(seq, **i32), S=max(1, max(seq)), Q=max(q), T=T,
               cu=torch.tensor([0] + list(np.cumsum(q)), **i32),
               q=(2 * torch.randn(T, case["Hq"], D, device=DEV, generator=g)).to(dt), out=torch.empty(T, case["Hq"], D, dtype=dt, device=DEV),
               lse=torch.empty(T, case["Hq"], device=DEV) if case["lse"] else None, scale=1 / math.sqrt(D))
    if own:
        import exact_lloyd_means_amd as fk
        st["ws"] = fk.kv4_attention_workspace(st["q"], st["seq"], st["codes"], st["Q"])
    return st


# ---- the operators in plain form -----------------------------------------------

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


def _plan(st):
    ctx, new, P, table, free, n = st["ctx"].long(), st["new"].long(), st["P"], st["table"], st["free"], st["count"].long()
    B, M = table.shape
    cap = st["slots"].numel()
    seq, old = ctx + new, (ctx + P - 1) // P
    need = ((seq + P - 1) // P).clamp(max=M).sub(old).clamp(min=0)
    off = need.cumsum(0) - need
    cu = torch.cat((seq.new_zeros(1), new.cumsum(0)))
    total, wanted = cu[-1], need.sum()
    taken = torch.minimum(wanted, n[0])
    page = torch.arange(M, device=DEV)
    i = n - 1 - (off[:, None] + page - old[:, None])
    fresh = (page >= old[:, None]) & (page < (old + need)[:, None])
    table[:] = torch.where(fresh, torch.where(i >= 0, free[i.clamp(0, free.numel() - 1)], -1), table)
    t = torch.arange(cap, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    pos = ctx[b] + t - cu[b]
    at = table[b, (pos // P).clamp(0, M - 1)]
    slots = torch.where((t < total) & (pos // P < M) & (at >= 0), at * P + pos % P, -1)
    got = (n - off).clamp(min=0).minimum(need)
    lost = (seq - ctx.maximum((old.clamp(max=M) + got) * P)).clamp(min=0).sum()
    status = torch.stack((total, taken, wanted - taken, lost))
    return {"table": table, "seq": seq.int(), "cu": cu.int(), "slots": slots.int(), "pos": torch.where(t < total, pos, -1).int(),
            "left": (n - taken).int(), "status": status.int()}


def _encode(x, cb):
    """Rows (T, H, D) -> codes and scales; cb (H, 16)."""
    x = x.float()
    scale = x.abs().amax(-1)
    scale = torch.where(scale < math.inf, scale, math.nan)
    mid = ((cb[:, :-1].float() + cb[:, 1:].float()) / 2).half().float()
    return (x[..., None] > (mid * scale[..., None])[:, :, None]).sum(-1, dtype=torch.uint8), scale


def _append(st):
    codes, scales, D, H = st["codes"], st["scales"], st["k"].shape[-1], st["k"].shape[1]
    P, dt = scales.shape[-1], scales.dtype
    keep = st["slots"] >= 0
    slot = st["slots"].long().clamp(min=0)
    heads = torch.arange(H, device=DEV)
    got = []
    ks = (_rows(torch.arange(16 * D, device=DEV), D, 0), _rows(torch.arange(16 * D, device=DEV), D, 1))
    row = ((slot // P)[:, None] * H + heads) * 2
    for kv, x in enumerate((st["k"], st["v"])):
        c, s = _encode(x, st["cb"][kv])
        block = (row + kv) * (P // 32) + (slot % P // 32)[:, None]
        at = block[..., None] * (16 * D) + ks[kv][slot % 32][:, None]
        codes.view(-1)[at[keep]] = (c[..., ::2] | c[..., 1::2] << 4)[keep]
        scales.view(-1)[((row + kv) * P + (slot % P)[:, None])[keep]] = s[keep].to(dt)
        back = codes.view(-1)[at].transpose(0, 1)
        s = scales.view(-1)[(row + kv) * P + (slot % P)[:, None]].transpose(0, 1)
        got.append(torch.where(keep[:, None, None], _values(back, s, st["cb"][kv]).transpose(0, 1), 0).to(dt))
    return {"k": got[0], "v": got[1]}


def _attend(st):
    c = st["case"]
    D, H, P = c["D"], c["Hkv"], c["P"]
    B, G, Q, M = c["B"], c["Hq"] // c["Hkv"], st["Q"], st["table"].shape[1]
    table = st["table"].clamp(min=0).long()
    # k, v (B, H, S, D) in float32
    k, v = (_values(_rows(st["codes"][:, :, kv][table], D, kv).permute(0, 2, 1, 3, 4, 5).reshape(B, H, M * P, D // 2),
                    st["scales"][:, :, kv][table].transpose(1, 2).reshape(B, H, M * P), st["cb"][kv]) for kv in (0, 1))
    cu, seq = st["cu"].long(), st["seq"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=DEV)
    there = i < n[:, None]
    at = torch.where(there, cu[:-1, None] + i, 0)
    q = st["q"].float()[at].view(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    s = (q @ k.transpose(-1, -2) * st["scale"]).view(B, H, G, Q, M * P)
    pos = (seq - n)[:, None, None] + i[:, None]
    j = torch.arange(M * P, device=DEV)
    seen = j < seq[:, None, None]
    if c["causal"]:
        seen = seen & (j <= pos)
    if c["window"]:
        seen = seen & (j > pos - c["window"])
    seen = seen[:, None, None]
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, 0))
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0]
    o = (p / torch.where(total > 0, total, 1)).view(B, H, G * Q, M * P) @ v
    o = o.view(B, H, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, H * G, D)[there]
    lse = lse.permute(0, 3, 1, 2).reshape(B, Q, H * G)[there]
    return {"out": o.to(st["q"].dtype), "lse": lse if c["lse"] else None}


def run(st):
    if not own:
        return {"plan": _plan, "append": _append, "attend": _attend}[st["kind"]](st)
    import exact_lloyd_means_amd as fk
    if st["kind"] == "plan":
        fk.fk_kv_plan(st["ctx"], st["new"], st["P"], st["free"], st["count"], st["table"], st["seq"], st["cu"], st["slots"],
                      st["pos"], st["left"], st["status"], ws=st["ws"])
        return {k: st[k] for k in ("table", "seq", "cu", "slots", "pos", "left", "status")}
    if st["kind"] == "append":
        fk.fk_kv4_write(st["k"], st["v"], st["slots"], st["cb"], st["codes"], st["scales"])
        fk.fk_kv4_read(st["slots"], st["cb"], st["codes"], st["scales"], st["ko"], st["vo"])
        return {"k": st["ko"], "v": st["vo"]}
    c = st["case"]
    fk.fk_kv4_attention(st["q"], st["cu"], st["seq"], st["table"], st["cb"], st["codes"], st["scales"], st["out"], st["Q"],
                        scale=st["scale"], causal=c["causal"], window=c["window"], lse=st["lse"], ws=st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


# ---- the definitions in 64 bits ---------------------------------------------------

def _address(D, kv):
    """Byte and shift of the code of (token t of a block, dimension d), from the layout's definition."""
    t, d = np.meshgrid(np.arange(32), np.arange(D), indexing="ij")
    if kv == 0:                                     # a lane (16 g + m) holds D/4 dimensions of two tokens
        m, tile, g, w = 4 * (t // 8) + t % 4, t // 4 % 2, d // (D // 4), d % (D // 4)
        at = tile * (D // 8) + w // 2               # the lane's byte
        lane = 16 * g + m
    else:                                           # a lane (16 g + r) holds D/16 dimensions of eight tokens
        g, j, r, w = t // 8, t % 8, d // (D // 16), d % (D // 16)
        at = (w // 8) * 32 + j * min(4, D // 32) + w % 8 // 2
        lane = 16 * g + r
    return torch.from_numpy(at // 16 * 1024 + lane * 16 + at % 16).to(DEV), torch.from_numpy(d % 2 * 4).to(DEV)


def exact(case, seed):
    if case["kind"] == "plan":
        return None
    st = prepare(case, seed)
    D, P, H = case["D"], case["P"], case["Hkv"]
    cb = st["cb"].double()
    if case["kind"] == "append":
        keep, got = (st["slots"] >= 0)[:, None, None], []
        for kv, x in enumerate((st["k"], st["v"])):
            x = x.double()
            s = x.abs().amax(-1, keepdim=True)
            mid = ((cb[kv, :, 1:] + cb[kv, :, :-1]) / 2).half().double()
            code = torch.zeros(x.shape, dtype=torch.int64, device=DEV)
            for j in range(15):
                code += mid[None, :, None, j] * s < x
            y = torch.gather(cb[kv][None].expand(x.shape[0], -1, -1), 2, code) * s
            got.append(torch.where(keep, y, 0))
        return {"k": got[0], "v": got[1]}
    if work(case)["flops"] > 3e12:
        return None
    outs, lses = [], []
    seq, cu, G = st["seq"].tolist(), st["cu"].tolist(), case["Hq"] // H
    place = [_address(D, kv) for kv in (0, 1)]
    for b, S in enumerate(seq):
        n = cu[b + 1] - cu[b]
        q = st["q"][cu[b]:cu[b + 1]].double().view(n, H, G, D)
        o = torch.zeros(n, H, G, D, dtype=torch.float64, device=DEV)
        lse = torch.full((n, H, G), -math.inf, dtype=torch.float64, device=DEV)
        first = max(0, S - n - case["window"]) // P * P if case["window"] else 0
        if S:
            j = torch.arange(first, S, device=DEV)
            page, t = st["table"][b].long()[j // P], j % P
            pos = torch.arange(S - n, S, device=DEV)[:, None]
            seen = torch.ones(n, len(j), dtype=torch.bool, device=DEV)
            seen &= j <= pos if case["causal"] else True
            seen &= j > pos - case["window"] if case["window"] else True
            for h in range(H):
                kv = []
                for w in (0, 1):
                    byte = torch.gather(st["codes"][page, h, w, t // 32], 1, place[w][0][t % 32])
                    kv.append(cb[w, h][(byte.int() >> place[w][1][t % 32] & 15).long()] * st["scales"][page, h, w, t].double()[:, None])
                for a in range(0, n, 512):
                    s = (q[a:a + 512, h].reshape(-1, D) @ kv[0].T * st["scale"]).view(-1, G, len(j))
                    s = s.masked_fill(~seen[a:a + 512, None], -math.inf)
                    l = torch.logsumexp(s, -1)
                    lse[a:a + 512, h] = l
                    p = torch.exp(s - torch.where(l > -math.inf, l, 0)[..., None])
                    o[a:a + 512, h] = (p.view(-1, len(j)) @ kv[1]).view(-1, G, D)
        outs.append(o.flatten(1, 2))
        lses.append(lse.flatten(1, 2))
    return {"out": torch.cat(outs), "lse": torch.cat(lses) if case["lse"] else None}
