"""Attention of requests that share a prefix against its 64-bit definition, which
reads every request's own row of the table."""
import math
import random

import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref
from test_gpu_streams import Bystanders, stall

pytestmark = pytest.mark.gpu
DT = ref.DT


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def problem(groups, alone, Hq, H, D, P, dtype, seed=0, copied=False, first=0, room=1 << 20):
    """Tables have room for so many tokens more than the longest request: how much
    of a prefix there may be decides whether it is walked once for all.  groups: (prefix tokens, [(tokens behind it, query tokens), ...]); alone: [(tokens, query tokens), ...].  copied: a
    prefix's last, partly filled page is a copy of the first request's; first: requests of no group before the groups."""
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    rows, cug, prefix = [], [], []
    for s, n in alone[:first]:
        rows.append(([], s, n))
    cug.append(len(rows))
    pages = 0
    copies = []
    for p, members in groups:
        whole, part = p // P, p % P if copied else 0
        shared = [("g", len(prefix), e) for e in range(whole)]
        for i, (s, n) in enumerate(members):
            rows.append((shared, (whole * P) + part + s, n))
            if part and i:
                copies.append((len(rows) - 1, whole, cug[-1]))
        prefix.append(whole * P + part)
        cug.append(len(rows))
    for s, n in alone[first:]:
        rows.append(([], s, n))
    need = sum(p // P for p, _ in groups) + sum(-(-s // P) for _, s, _ in rows) + 2
    ids = list(range(need))
    r.shuffle(ids)
    of = {}
    M = max([1] + [-(-s // P) for _, s, _ in rows]) + room // P
    table = torch.full((len(rows), M), -1, dtype=torch.int32)
    for b, (shared, s, _) in enumerate(rows):
        for e in range(-(-s // P)):
            if e < len(shared):
                if shared[e] not in of:
                    of[shared[e]] = ids.pop()
                table[b, e] = of[shared[e]]
            else:
                table[b, e] = ids.pop()
    codes = torch.randint(0, 256, (need, H, 2, P // 32, 16 * D), generator=g, dtype=torch.uint8)
    scales = (2 * torch.exp(0.4 * torch.randn(need, H, 2, P, generator=g))).to(dtype)
    for b, e, src in copies:
        codes[table[b, e].long()], scales[table[b, e].long()] = codes[table[src, e].long()], scales[table[src, e].long()]
    seq, n = [s for _, s, _ in rows], [n for _, _, n in rows]
    cu = [sum(n[:i]) for i in range(len(n) + 1)]
    q = (2 * torch.randn(cu[-1], Hq, D, generator=g)).to(dtype)
    return dict(q=q, cu=cu, seq=seq, table=table, cug=cug, prefix=prefix, cb=ref.codebook(H, seed), codes=codes, scales=scales)


def run(p, max_q, causal=True, window=0, lse=True, scale=None, stream=None, ws=None):
    dev = {k: v.cuda() for k, v in p.items() if isinstance(v, torch.Tensor)}
    out = torch.full(p["q"].shape, 7.0, dtype=p["q"].dtype, device="cuda")
    l = torch.full(p["q"].shape[:2], 7.0, device="cuda") if lse else None
    fk.fk_kv4_attention_shared(dev["q"], i32(p["cu"]), i32(p["seq"]), dev["table"], i32(p["cug"]), i32(p["prefix"]), dev["cb"],
                               dev["codes"], dev["scales"], out, max_q, scale=scale, causal=causal, window=window, lse=l,
                               stream=stream, ws=ws)
    torch.cuda.synchronize()
    return out, l


def check(p, max_q=None, causal=True, window=0, lse=True):
    D = p["q"].shape[-1]
    n = [b - a for a, b in zip(p["cu"], p["cu"][1:])]
    out, l = run(p, max_q or max(n + [1]), causal, window, lse)
    want = ref.attention(p["q"], p["cu"], p["seq"], p["table"], p["cb"], p["codes"], p["scales"], 1 / math.sqrt(D), causal, window)
    tol, ltol = ref.attention_tolerance(*want, D, p["q"].dtype)
    off = (out.cpu().double() - want[0]).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    if lse:
        same = (l.cpu().double() == want[1]) | ((l.cpu().double() - want[1]).abs() <= ltol)
        assert bool(same.all())
    return out, l


@pytest.mark.parametrize("Hq,H,D,P,dtype", [(8, 2, 128, 64, "bf16"), (8, 1, 64, 32, "f16"), (3, 3, 128, 96, "f16"), (4, 2, 256, 64, "bf16"),
                                            (24, 2, 64, 128, "bf16"), (5, 1, 256, 32, "f16")])
@pytest.mark.parametrize("q", [1, 3])
def test_matches_definition(Hq, H, D, P, dtype, q):
    groups = [(700, [(5 + i, q) for i in range(9)]), (P, [(200, q)] * 2), (2000, [(q, q), (70, q), (P, q)])]
    check(problem(groups, [(q, q), (300, q)], Hq, H, D, P, DT[dtype], seed=D + q))


@pytest.mark.parametrize("window", [1, 33, 500, 1900, 100000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(window, causal):
    groups = [(1024, [(1, 1), (900, 2), (40, 3), (333, 1)]), (640, [(2000, 4)] * 2)]
    check(problem(groups, [(50, 1)], 8, 2, 128, 64, DT["bf16"], seed=window), causal=causal, window=window)


def test_a_window_of_everything():
    # the largest that there is leaves nothing out, and is shared like none
    p = problem([(1024, [(1 + 17 * i, 1 + i % 3) for i in range(14)])], [(50, 1)], 16, 4, 128, 64, DT["f16"], seed=77)
    out, lse = check(p, window=2 ** 31 - 1)
    again, lse_again = run(p, 3)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


@pytest.mark.parametrize("window", [700, 1000, 1900])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_of_many_heads(window, causal):
    # so many that the window's blocks alone are worth sharing
    groups = [(1024, [(1 + 17 * i, 1 + i % 3) for i in range(14)]), (640, [(900 - 50 * i, 1) for i in range(14)])]
    check(problem(groups, [(50, 1)], 16, 16, 256, 64, DT["bf16"], seed=window), causal=causal, window=window)


@pytest.mark.parametrize("room", [0, 64])
def test_tables_without_room(room):
    # where little can be shared the requests are taken as if nothing were
    check(problem([(300, [(20, 1)] * 3)], [(9, 1)], 8, 2, 128, 32, DT["bf16"], seed=21, room=room))


@pytest.mark.parametrize("G,each,D", [(1, 2, 64), (1, 16, 128), (1, 33, 128), (5, 6, 64), (3, 40, 128), (12, 2, 256), (24, 2, 128), (32, 3, 64),
                                      (40, 2, 256), (33, 2, 128), (24, 8, 128), (20, 6, 64)])
def test_rows_of_all_kinds_of_tiles(G, each, D):
    check(problem([(500, [(1 + 3 * i, 1) for i in range(each)]), (96, [(40, 1)] * each)], [(70, 1)], 2 * G, 2, D, 32, DT["f16"], seed=G))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_long_prefix(D):
    # shares that lie within a tile, and many tiles of rows
    check(problem([(20000, [(i + 1, 1) for i in range(30)])], [], 16, 2, D, 64, DT["bf16"], seed=1))


@pytest.mark.parametrize("G,D,dtype", [(1, 64, "bf16"), (20, 64, "f16"), (7, 128, "bf16"), (2, 256, "f16")])
def test_long_own_keys_behind_short_prefixes(G, D, dtype):
    # segments end long before the requests' own keys do, whose rest their
    # workgroups take; a second call gives the same bits
    groups = [(96, [(700 + 37 * i, 1) for i in range(20)]), (64, [(1100, 1)] * 20), (128, [(1500 - 60 * i, 1) for i in range(20)])]
    p = problem(groups, [(900, 1), (3, 1)], 16 * G, 16, D, 32, DT[dtype], seed=90 + D + G, first=1, room=900)
    out, lse = check(p)
    again, lse_again = run(p, 1)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


def test_many_groups():
    # more requests than a workgroup has threads
    r = random.Random(4)
    groups = [(32 * r.randrange(0, 6), [(r.randrange(1, 60), 1) for _ in range(r.randrange(0, 7))]) for _ in range(110)]
    check(problem(groups, [(20, 1)] * 7, 4, 1, 64, 32, DT["f16"], seed=4, first=3))


def test_ragged_queries_and_empty_requests():
    groups = [(256, [(4, 4), (0, 0), (300, 1), (2, 2), (7, 0)]), (0, [(50, 2), (60, 1)]), (512, [])]
    check(problem(groups, [(0, 0), (0, 1), (3, 5), (100, 2)], 8, 2, 128, 64, DT["bf16"], seed=5, first=2))


def test_queries_within_the_prefix():
    # requests whose own tokens are part of what is shared, or that are shorter than it
    p = problem([(320, [(0, 3), (1, 5), (40, 2)])], [], 8, 2, 128, 32, DT["bf16"], seed=6)
    check(p)
    p["seq"][1] = 100
    check(p)
    check(p, causal=False)


def test_prefix_ends_within_a_page():
    # 100 tokens: 96 of them in whole blocks, in a page that the others hold as copies
    check(problem([(100, [(3, 1)] * 5), (95, [(1, 1)] * 3)], [], 8, 2, 128, 64, DT["f16"], seed=7, copied=True))


def test_max_q_leaves_tokens_out():
    p = problem([(300, [(20, 1), (30, 6), (9, 2)])], [(40, 5)], 8, 2, 128, 32, DT["bf16"], seed=8)
    out, l = run(p, 2)
    want, _ = run(p, 6)
    for b, (a, e) in enumerate(zip(p["cu"], p["cu"][1:])):
        assert bool((out[a + 2:e] == 7).all()) and bool((l[a + 2:e] == 7).all())
    kept = torch.tensor([i for a, e in zip(p["cu"], p["cu"][1:]) for i in range(a, min(e, a + 2))])
    # the positions of kept tokens do not change
    tol = 2.0 ** -7 * want.float().abs().amax(-1, keepdim=True) + 2.0 ** -6
    assert bool(((out.float() - want.float()).abs() <= tol)[kept].all())


def test_rows_behind_the_last_request():
    p = problem([(300, [(20, 1), (30, 1)])], [], 8, 2, 128, 32, DT["bf16"], seed=9)
    p["q"] = torch.cat((p["q"], p["q"]))
    out, l = run(p, 1)
    assert bool((out[2:] == 7).all()) and bool((l[2:] == 7).all()) and not bool((out[:2] == 7).all())


def test_odd_numbers_in_pages():
    # scales that are infinite or NaN where nobody looks; pages that are missing; groups that are none
    p = problem([(128, [(40, 1), (70, 1)]), (64, [(9, 1)])], [(33, 1)], 8, 2, 128, 32, DT["bf16"], seed=10)
    named = set(p["table"].flatten().tolist())
    for page in range(len(p["codes"])):
        if page not in named:
            p["scales"][page] = math.nan
    p["scales"][p["table"][0, 5].long(), :, :, 8:] = math.nan           # behind the 168 tokens of the first request
    p["scales"][p["table"][1, 6].long(), :, :, 6:] = math.inf
    check(p)
    p["table"][:2, 1] = -1                                              # 32 tokens of the prefix
    p["table"][3, 0] = 10 ** 6
    check(p)
    # bounds beyond the requests; the second group's two have nothing in common, which is said by a prefix of none
    p["cug"], prefix, p["prefix"] = [-3, 2, 100], p["prefix"], [128, 0]
    check(p)
    p["prefix"] = prefix
    for cug in ([2, 0, 3], [0, 4, 1], [0, 2, 1]):                       # lists that descend share nothing
        p["cug"] = cug
        check(p)
    p["cug"], p["prefix"] = [0, 2, 3], [-5, 10 ** 9]
    p["seq"][2] = 73
    check(p)


def test_query_lists_that_descend():
    # tokens named by no ascending list: no row is written twice, none beyond the buffers; ascending requests are right
    p = problem([(128, [(40, 1)] * 4), (96, [(9, 1)] * 4)], [(30, 1)], 4, 1, 128, 32, DT["bf16"], seed=20)
    want, _ = run(p, 1)
    p["cu"] = [0, 1, 2, 3, 1, 5, 6, 7, 8, 9]                            # request 3 has no tokens, request 4 those from 1 on
    out, _ = run(p, 4)
    # two roundings to bf16, and of the weights to fp16 (2 2^-11 of values up to 10)
    assert bool(((out[5:].float() - want[5:].float()).abs() <= 2.0 ** -7 * want[5:].float().abs() + 10 * 2.0 ** -10).all())


def test_same_bits_every_time():
    p = problem([(3000, [(100 + i, 1) for i in range(20)])], [(500, 1)], 8, 2, 128, 64, DT["bf16"], seed=11)
    a, la = run(p, 1)
    for _ in range(3):
        b, lb = run(p, 1)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_strided_queries():
    p = problem([(500, [(20, 1), (30, 1), (2, 1)])], [], 8, 2, 64, 32, DT["bf16"], seed=12)
    want, _ = run(p, 1)
    whole = torch.zeros(3, 13, 67, dtype=torch.bfloat16)
    whole[:, 3:11, 1:65] = p["q"]
    q = whole.cuda()[:, 3:11, 1:65]
    out = torch.empty_like(want)
    fk.fk_kv4_attention_shared(q, i32(p["cu"]), i32(p["seq"]), p["table"].cuda(), i32(p["cug"]), i32(p["prefix"]), p["cb"].cuda(),
                               p["codes"].cuda(), p["scales"].cuda(), out, 1)
    assert torch.equal(out, want)


def test_workspace_on_another_stream():
    p = problem([(2000, [(100 + i, 1) for i in range(20)])], [], 8, 2, 128, 64, DT["bf16"], seed=13)
    want, _ = run(p, 1)
    dev = {k: v.cuda() for k, v in p.items() if isinstance(v, torch.Tensor)}
    args = (dev["q"], i32(p["cu"]), i32(p["seq"]), dev["table"], i32(p["cug"]), i32(p["prefix"]), dev["cb"], dev["codes"], dev["scales"])
    out, side = torch.zeros_like(want), torch.cuda.Stream()
    size = fk.kv4_attention_shared_workspace(dev["q"], args[2], args[5], dev["codes"], 1).numel()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stall(side)
    fk.fk_kv4_attention_shared(*args, out, 1, stream=side)
    assert Bystanders([size]).untouched()
    assert torch.equal(out, want)


def test_captured():
    p = problem([(1000, [(100 + i, 1) for i in range(6)])], [(300, 1)], 8, 2, 128, 64, DT["bf16"], seed=14)
    dev = {k: v.cuda() for k, v in p.items() if isinstance(v, torch.Tensor)}
    cu, seq, cug, prefix = i32(p["cu"]), i32(p["seq"]), i32(p["cug"]), i32(p["prefix"])
    out = torch.empty(p["q"].shape, dtype=torch.bfloat16, device="cuda")
    ws = fk.kv4_attention_shared_workspace(dev["q"], seq, prefix, dev["codes"], 1)
    args = (dev["q"], cu, seq, dev["table"], cug, prefix, dev["cb"], dev["codes"], dev["scales"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fk.fk_kv4_attention_shared(*args, out, 1, ws=ws)
    for i in range(3):
        seq += -7 * i
        prefix += -64 * i
        ws.fill_(255)
        graph.replay()
        want = torch.empty_like(out)
        fk.fk_kv4_attention_shared(*args, want, 1)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
