"""The 4-bit paged cache on the GPU against its 64-bit definition."""
import math
import random

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- plan ---------------------------------------------------------------------

def run_plan(ctx, new, P, M, free, count, cap, positions=True, alias=False, stream=None):
    B = len(ctx)
    r = random.Random(B + P)
    table = [[r.randrange(1000, 9000) if p < -(-max(0, c) // P) else -7 for p in range(M)] for c in ctx]
    tab = i32(table)
    cnt = i32([count])
    seq, cu = i32([-5] * B), i32([-5] * (B + 1))
    slots, pos = i32([-5] * cap), i32([-5] * cap)
    left = cnt if alias else i32([-5])
    status = i32([-5] * 4)
    fk.fk_kv_plan(i32(ctx), i32(new), P, i32(free), cnt, tab, seq, cu, slots,
                  pos if positions else None, left, status, stream=stream)
    torch.cuda.synchronize()
    want = ref.plan(ctx, new, P, table, free, count, cap)
    assert tab.cpu().tolist() == table
    assert seq.cpu().tolist() == want["seq"]
    assert cu.cpu().tolist() == want["cu"]
    assert slots.cpu().tolist() == want["slots"]
    if positions:
        assert pos.cpu().tolist() == want["pos"]
    else:
        assert pos.cpu().tolist() == [-5] * cap
    assert left.item() == want["left"]
    assert status.cpu().tolist() == want["status"]


@pytest.mark.parametrize("B,P,cap_more", [(1, 32, 0), (3, 96, 5), (64, 64, 0), (257, 32, 100),
                                          (1000, 1024, 20000), (4096, 32, 3), (4097, 64, 0),
                                          (9000, 32, 77)])
def test_plan_matches_definition(B, P, cap_more):
    r = random.Random(B * 7 + P)
    ctx = [r.choice([0, 1, P - 1, P, P + 1, r.randrange(0, 5 * P)]) for _ in range(B)]
    new = [r.choice([0, 1, 1, 1, 2, P, r.randrange(0, 2 * P)]) for _ in range(B)]
    need = sum(-(-(c + n) // P) for c, n in zip(ctx, new))
    free = list(range(20000, 20000 + need + 3))
    run_plan(ctx, new, P, 9, free, len(free), max(1, sum(new) + cap_more))


@pytest.mark.parametrize("B", [40, 5000])      # one and two launches
def test_plan_when_list_or_table_ends(B):
    r = random.Random(B)
    P, M = 32, 4
    ctx = [r.randrange(0, 100) for _ in range(B)]
    new = [r.randrange(0, 90) for _ in range(B)]
    total = sum(new)
    for count, nfree in ((B // 2, B), (0, 5), (-3, 5), (B, B // 3)):
        run_plan(ctx, new, P, M, list(range(100, 100 + nfree)), count, total, alias=True)
    # fewer slots than tokens: the tables are filled all the same
    run_plan(ctx, new, P, M, list(range(100, 100 + 9 * B)), 9 * B, total // 3, positions=False)
    # contexts beyond the table, negative lengths, nothing new
    run_plan([200] * B, [70] * B, P, M, list(range(9)), 9, 70 * B)
    run_plan([-4] * B, [-1] * B, P, M, list(range(9)), 9, 7)
    run_plan([0] * B, [0] * B, P, M, [], 0, 1)


def test_plan_long_prompt_two_launches_on_a_side_stream():
    side = torch.cuda.Stream()
    run_plan([5, 0, 33], [30001, 0, 1], 64, 600, list(range(50000, 51000)), 1000, 30100, stream=side)


# ---- rows ---------------------------------------------------------------------

def make_cache(pages, H, D, P, dtype, seed=0, cb=None):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (pages, H, 2, P // 32, 16 * D), dtype=torch.uint8, generator=g)
    scales = (2.7 * torch.exp(0.4 * torch.randn(pages, H, 2, P, generator=g))).to(DT[dtype])
    cb = ref.codebook(H, seed) if cb is None else cb
    return codes, scales, cb


def check_rows(k, v, slots, cache):
    """Writes k, v and compares every byte and scale of the cache, then reads."""
    codes, scales, cb = (t.clone() for t in cache)
    P, D, H = scales.shape[3], codes.shape[4] // 16, codes.shape[1]
    gc, gs, gb = codes.cuda(), scales.cuda(), cb.cuda()
    sl = slots.cuda()
    fk.fk_kv4_write(k, v, sl, gb, gc, gs)
    T = len(slots)
    ko, vo = (torch.full((T, H, D), 7.0, dtype=scales.dtype, device="cuda") for _ in range(2))
    fk.fk_kv4_read(sl, gb, gc, gs, ko, vo)
    torch.cuda.synchronize()
    n = codes.shape[0] * P
    for kv, x in enumerate((k.cpu(), v.cpu())):
        c, s = ref.encode(x, cb[kv])
        at, sh = ref.place_tables(D, kv)
        for t in range(T):
            slot = int(slots[t])
            if slot < 0 or slot >= n:
                continue
            page, i = slot // P, slot % P
            for h in range(H):
                row = codes[page, h, kv, i // 32]
                b = c[t, h, ::2] | c[t, h, 1::2] << 4
                row[at[i % 32][::2]] = b
                scales[page, h, kv, i] = s[t, h].to(scales.dtype)
    assert torch.equal(gc.cpu(), codes)
    a, b = gs.cpu(), scales
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(torch.nan_to_num(a.double()), torch.nan_to_num(b.double()))
    # the rows read are the definition's values rounded once
    good = (slots >= 0) & (slots < n)
    sl = slots.long().clamp(0, n - 1)
    want = ref.gather(codes, scales, cb, sl // P, sl % P)
    want = torch.where(good[None, :, None, None], want, 0.0).to(scales.dtype)
    for got, w in zip((ko.cpu(), vo.cpu()), want):
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(torch.nan_to_num(got.double()), torch.nan_to_num(w.double()))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,P", [(1, 1, 32), (37, 3, 96), (130, 2, 64)])
def test_write_and_read_rows(dtype, D, T, H, P):
    g = torch.Generator().manual_seed(T * D)
    cache = make_cache(T // P + 4, H, D, P, dtype, seed=T)
    n = cache[0].shape[0] * P
    slots = torch.randperm(n, generator=g)[:T].int()
    if T > 8:
        slots[3], slots[5], slots[7] = -1, n, 2 ** 31 - 1
    k, v = (torch.randn(T, H, D, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    check_rows(k, v, slots, cache)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rows_at_the_ends_of_the_type(dtype):
    H, D, P = 2, 64, 32
    big = torch.finfo(DT[dtype]).max
    cb = ref.codebook(H, 4)
    cb[0, 0, 3:9] = cb[0, 0, 3]                  # equal values: thresholds coincide
    cb[1, 1] = 0.25                              # a codebook of one value
    cache = make_cache(2, H, D, P, dtype, 1, cb)
    x = torch.randn(16, H, D, generator=torch.Generator().manual_seed(3))
    x[0] = 0
    x[1] = big
    x[2, :, ::2] = -big
    x[3, :, 5] = math.inf
    x[4, :, 6] = -math.inf
    x[5, :, 7] = math.nan
    x[6] = torch.finfo(DT[dtype]).tiny / 4       # below the normal range
    x[7, :, 1:] = 0
    x[8] = -0.0
    # values on the thresholds themselves: the lower code
    t = ((cb[..., :-1].double() + cb[..., 1:].double()) / 2).half().double()
    x[9, :, :15] = t[0].float()
    x[9, :, 15:] = 1.0
    x = x.to(DT[dtype]).cuda()
    check_rows(x, x.flip(0).contiguous(), torch.randperm(64, generator=torch.Generator().manual_seed(1))[:16].int(),
               cache)


@pytest.mark.parametrize("off", [0, 1, 4, 8])    # elements: rows aligned to 2, 8 and 16 bytes
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_a_fused_projection(off, D):
    H, Hq, T, P = 2, 3, 21, 32
    g = torch.Generator().manual_seed(off)
    buf = torch.randn(T, (Hq + 2 * H) * D + 16, generator=g).to(torch.float16).cuda()
    k = buf[:, off + Hq * D:][:, :H * D].unflatten(1, (H, D))
    v = buf[:, off + (Hq + H) * D:][:, :H * D].unflatten(1, (H, D))
    check_rows(k, v, torch.randperm(64, generator=g)[:T].int(), make_cache(2, H, D, P, "f16", 5))
    # heads first, tokens last
    kt = torch.randn(H, T, D, generator=g).to(torch.float16).cuda().transpose(0, 1)
    check_rows(kt, kt, torch.randperm(64, generator=g)[:T].int(), make_cache(2, H, D, P, "f16", 6))


def test_many_heads_beyond_static_lds():
    H, D, P = 700, 64, 32
    g = torch.Generator().manual_seed(2)
    cache = make_cache(1, H, D, P, "bf16", 3)
    x = torch.randn(2, H, D, generator=g).to(torch.bfloat16).cuda()
    check_rows(x, -x, torch.tensor([31, 0], dtype=torch.int32), cache)


# ---- attention ------------------------------------------------------------------

def attention_case(seq, qlen, Hq, H, D, P, dtype, causal=True, window=0, seed=0, spoil=None, extra=0,
                   q=None, scale=None, pages_more=2, stream=None, max_q=None):
    g = torch.Generator().manual_seed(seed)
    B = len(seq)
    held = [-(-s // P) for s in seq]
    M = max(1, max(held)) + extra
    pages = sum(held) + pages_more
    ids = torch.randperm(pages, generator=g).int()
    table = torch.full((B, M), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    codes, scales, cb = make_cache(pages, H, D, P, dtype, seed)
    cu = torch.tensor([0] + list(np.cumsum(qlen)), dtype=torch.int32)
    T = int(cu[-1])
    if q is None:
        q = (2 * torch.randn(T, Hq, D, generator=g)).to(DT[dtype])
    if spoil:
        spoil(codes, scales, table, seq)
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    dev = [t.cuda() for t in (cu, torch.tensor(seq, dtype=torch.int32), table, cb, codes, scales)]
    qd = q.cuda() if q.device.type == "cpu" else q
    torch.cuda.synchronize()
    fk.fk_kv4_attention(qd, *dev, out, max_q or max(qlen), scale=scale, causal=causal, window=window,
                        lse=lse, stream=stream)
    torch.cuda.synchronize()
    want = ref.attention(q.cpu(), cu, seq, table, cb, codes, scales, scale, causal, window)
    check_attention(out.cpu(), lse.cpu(), want, D)
    return out, lse


def check_attention(out, lse, want, D):
    o, l, pv, dot, svmax = want
    tol, tol_lse = ref.attention_tolerance(o, l, pv, dot, svmax, D, out.dtype)
    nan = torch.isnan(o)
    assert torch.equal(torch.isnan(out), nan), "NaN in other places"
    err = torch.where(nan, 0.0, (out.double() - torch.where(nan, 0.0, o)).abs())
    tol = torch.where(nan, 1.0, tol)
    assert bool((err <= tol).all()), f"out: {float((err / tol).max())} times the tolerance"
    empty = l == -math.inf
    assert bool((lse[empty] == -math.inf).all()) and bool((out[empty] == 0).all())
    ok = torch.isfinite(l)
    assert torch.equal(torch.isfinite(lse), ok)
    e = (lse.double() - l)[ok].abs()
    assert bool((e <= tol_lse[ok]).all()), f"lse: {float((e / tol_lse[ok]).max())} times the tolerance"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(1, 1), (6, 2), (8, 1), (17, 1), (40, 1), (80, 1)])
def test_single_tokens(dtype, D, Hq, H):
    seq = [1, 2, 31, 32, 33, 64, 65, 129, 0, 300, 1000]
    attention_case(seq, [1] * len(seq), Hq, H, D, 64, dtype, seed=D + Hq)


@pytest.mark.parametrize("dtype,D,P", [("f16", 64, 32), ("bf16", 128, 96), ("f16", 256, 128), ("bf16", 64, 1024)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 40, 5000])
def test_few_and_many_query_tokens(dtype, D, P, causal, window):
    # more query tokens than positions: the first rows see nothing
    seq = [5, 64, 100, 257, 700, 0, 90, 1]
    qlen = [9, 64, 1, 33, 120, 3, 0, 1]
    attention_case(seq, qlen, 6, 2, D, P, dtype, causal, window, seed=window + D)
    attention_case(seq, [min(n, 4) for n in qlen], 6, 2, D, P, dtype, causal, window, seed=window)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16"), (256, "bf16")])
@pytest.mark.parametrize("window", [0, 100])
def test_prompts_that_fill_the_card(D, dtype, window):
    # enough rows for one wave a row tile; ragged, one request behind a context
    H, Hq = 16, 64
    attention_case([701, 1300, 64, 900], [701, 517, 64, 900], Hq, H, D, 64, dtype, True, window, seed=D)


@pytest.mark.parametrize("dtype,D", [("f16", 64), ("bf16", 64), ("f16", 128), ("bf16", 128), ("f16", 256), ("bf16", 256)])
@pytest.mark.parametrize("Hq,qlen", [(4, [1, 1, 1, 1, 1, 1]), (12, [3, 1, 0, 4, 2, 5]), (14, [5, 6, 1, 7, 2, 5])])
@pytest.mark.parametrize("window", [0, 200])
def test_shares_of_the_keys(dtype, D, Hq, qlen, window):
    # a wide table: the keys are cut into equal shares whatever the lengths
    attention_case([700, 33, 0, 1500, 64, 5], qlen, Hq, 2, D, 32, dtype, True, window, seed=D + Hq, extra=100)


@pytest.mark.parametrize("dtype,D,P", [("f16", 128, 32), ("bf16", 256, 64), ("bf16", 64, 96)])
def test_many_short_requests_of_several_rows(dtype, D, P):
    # a wave a request and row tile
    r = random.Random(D)
    seq = [r.choice([0, 1, 31, 40, 200, 600]) for _ in range(180)]
    attention_case(seq, [r.choice([1, 2, 5]) for _ in seq], 24, 3, D, P, dtype, True, r.choice([0, 70]), seed=D)


@pytest.mark.parametrize("B,D,top", [(200, 64, 300), (200, 128, 640), (300, 128, 1200), (100, 256, 300)])
def test_groups_of_two_and_four_waves(B, D, top):
    r = random.Random(B + D)
    seq = [r.choice([0, 1, 33, r.randrange(2, top)]) for _ in range(B)]
    seq[B // 2] = top
    attention_case(seq, [r.choice([1, 1, 3]) for _ in seq], 8, 4, D, 32, "f16", True, 0, seed=B)


def test_more_prompts_than_the_order_sorts():
    r = random.Random(4)
    seq = [r.randrange(20, 120) for _ in range(300)]
    attention_case(seq, [s - r.choice([0, 0, 9]) for s in seq], 32, 8, 64, 32, "bf16", seed=2)


def test_one_request_is_split_over_the_card():
    attention_case([20011], [1], 4, 1, 128, 64, "bf16", seed=1)
    attention_case([9001, 3], [2, 1], 40, 1, 256, 32, "f16", seed=2)
    attention_case([9001, 3, 5000], [30, 1, 7], 8, 2, 64, 96, "f16", True, 3000, seed=3)


def test_many_requests():
    r = random.Random(5)
    seq = [r.choice([0, 1, 5, 40, 100]) for _ in range(700)]
    attention_case(seq, [1] * 700, 8, 2, 64, 32, "bf16", seed=9)


def test_max_q_may_be_larger():
    attention_case([100, 50], [3, 1], 4, 2, 64, 32, "f16", max_q=500)
    attention_case([100, 50], [3, 1], 4, 2, 128, 32, "f16", max_q=1 << 30)


def test_scales_after_the_last_token_do_not_matter():
    def spoil(codes, scales, table, seq):
        P = scales.shape[3]
        for b, s in enumerate(seq):
            if s % P:
                scales[int(table[b, s // P]), :, :, s % P:] = math.nan
        used = set(table.flatten().tolist())
        for p in range(scales.shape[0]):
            if p not in used:
                scales[p] = math.inf
    for q in ([1] * 6, [4, 1, 2, 30, 70, 1]):
        attention_case([1, 30, 33, 95, 200, 64], q, 4, 2, 128, 64, "bf16", spoil=spoil)


def test_pages_the_table_does_not_name():
    def spoil(codes, scales, table, seq):
        table[0, 1] = -1
        table[1, 0] = codes.shape[0]
        table[2, 2:] = 2 ** 31 - 1
        scales[0] = math.nan                     # the page a careless read would fall on
        table[table == 0] = codes.shape[0] - 1
    attention_case([200, 40, 300], [1, 1, 1], 4, 2, 64, 64, "f16", spoil=spoil)
    attention_case([200, 40, 300], [50, 7, 40], 4, 2, 128, 32, "f16", spoil=spoil)
    attention_case([200, 40, 300], [50, 7, 40], 4, 2, 256, 32, "bf16", True, 60, spoil=spoil)


@pytest.mark.parametrize("kv", [0, 1])
def test_nan_rows_reach_only_those_who_see_them(kv):
    def spoil(codes, scales, table, seq):
        scales[int(table[0, 2]), 0, kv, 3] = math.nan      # position 67 of request 0, kv head 0
    out, _ = attention_case([90, 80], [40, 3], 4, 2, 64, 32, "f16", spoil=spoil)
    # query i of request 0 stands at 50 + i: rows before 67 are finite
    bad = torch.isnan(out.float()).flatten(1)
    assert not bool(bad[:17].any()) and not bool(bad[40:].any())
    assert bool(torch.isnan(out[17:40, :2].float()).all()) and not bool(torch.isnan(out[:, 2:].float()).any())
    attention_case([90, 80], [40, 3], 4, 2, 64, 32, "f16", True, 20, spoil=spoil)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_and_small_magnitudes(dtype):
    # q rows and v scales of very different magnitudes, a very large score
    D, T = 128, 6
    q = torch.randn(T, 4, D, generator=torch.Generator().manual_seed(8))
    q[0] *= 1e-4
    q[1] *= 100
    q[2] = 0
    q[3, :, 0] = 3e4

    def spoil(codes, scales, table, seq):
        f = torch.tensor([1e-4, 1.0, 1e3, 3e-2, 40.0])[torch.arange(scales.shape[3]) % 5]
        scales[:, :, 1] = f.to(scales.dtype)
    attention_case([300, 200], [3, 3], 4, 2, D, 32, dtype, spoil=spoil, q=q.to(DT[dtype]))

    def tiny(codes, scales, table, seq):
        scales[:, :, 1] = 6e-8 if dtype == "f16" else 1e-30
        scales[:, :, 1, ::3] = 0
    attention_case([300, 200], [3, 3], 4, 2, D, 32, dtype, spoil=tiny)

    def zeros(codes, scales, table, seq):
        scales[:] = 0
    out, lse = attention_case([300, 200], [3, 3], 4, 2, D, 32, dtype, spoil=zeros)
    assert bool((out == 0).all())


def test_other_scale():
    attention_case([300], [2], 4, 2, 64, 32, "f16", scale=3.0)
    attention_case([300], [2], 4, 2, 64, 32, "f16", scale=1e-3)


@pytest.mark.parametrize("off", [0, 1, 8])
def test_queries_of_a_fused_projection(off):
    Hq, H, D, T = 4, 2, 128, 5
    buf = torch.randn(T, (Hq + 2 * H) * D + 16, generator=torch.Generator().manual_seed(1)).half().cuda()
    q = buf[:, off:off + Hq * D].unflatten(1, (Hq, D))
    attention_case([100, 50], [3, 2], Hq, H, D, 32, "f16", q=q)


def test_results_do_not_depend_on_timing():
    outs = [attention_case([5000, 900, 33], [2, 40, 1], 8, 2, 128, 64, "bf16", seed=4) for _ in range(3)]
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])


def test_side_stream():
    side = torch.cuda.Stream()
    attention_case([500, 90], [1, 1], 8, 2, 128, 64, "bf16", stream=side)


def test_offsets_beyond_32_bits():
    # 4.9 GB of codes; the last pages hold the rows
    pages, H, D, P = 600_000, 1, 128, 64
    cb = ref.codebook(H, 1)
    codes = torch.empty(pages, H, 2, P // 32, 16 * D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, H, 2, P, dtype=torch.float16, device="cuda")
    first = pages - 2
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(100, H, D, generator=g).half() for _ in range(2))
    slots = torch.arange(first * P, first * P + 100, dtype=torch.int32)
    assert first * codes[0].numel() > 2 ** 32
    fk.fk_kv4_write(k.cuda(), v.cuda(), slots.cuda(), cb.cuda(), codes, scales)
    ko, vo = (torch.empty(100, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    fk.fk_kv4_read(slots.cuda(), cb.cuda(), codes, scales, ko, vo)
    q = torch.randn(1, 4, D, generator=g).half()
    out = torch.empty(1, 4, D, dtype=torch.float16, device="cuda")
    lse = torch.empty(1, 4, device="cuda")
    fk.fk_kv4_attention(q.cuda(), i32([0, 1]), i32([100]), i32([[first, first + 1]]), cb.cuda(), codes, scales,
                        out, 1, lse=lse)
    torch.cuda.synchronize()
    small_c, small_s = codes[first:].cpu(), scales[first:].cpu()
    want = ref.gather(small_c, small_s, cb, torch.arange(100) // P, torch.arange(100) % P)
    assert torch.equal(ko.cpu(), want[0].half()) and torch.equal(vo.cpu(), want[1].half())
    c, s = ref.encode(k, cb[0])
    assert torch.equal(small_s[torch.arange(100) // P, :, 0, torch.arange(100) % P].double(), s)
    r = ref.attention(q, torch.tensor([0, 1]), [100], torch.tensor([[0, 1]], dtype=torch.int32), cb, small_c, small_s,
                      1 / math.sqrt(D), True, 0)
    check_attention(out.cpu(), lse.cpu(), r, D)
