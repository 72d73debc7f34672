"""KV4Cache with forks, drafts, rotated rows and compaction: what the rows hold is
what was written for them, and every page is in the list or in the table."""
import math
import random

import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref
import serve_ref
from test_gpu_streams import Bystanders, stall

pytestmark = pytest.mark.gpu
H, Hq, D, P = 2, 4, 64, 32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Serving:
    """A cache beside what its rows should hold."""

    def __init__(self, pages, R, seed=0):
        self.cache = fk.KV4Cache(pages, P, H, D, ref.codebook(H, 0).cuda(), R, 400)
        self.k, self.v = ([torch.empty(0, H, D, dtype=torch.bfloat16) for _ in range(R)] for _ in range(2))
        self.g, self.R, self.pages = torch.Generator().manual_seed(seed), R, pages

    def step(self, new, shared=None):
        total, R = sum(new), self.R
        self.cache.plan(i32(new), total)
        q, k, v = (torch.randn(total, h, D, generator=self.g).bfloat16() for h in (Hq, H, H))
        self.cache.append(k.cuda(), v.cuda())
        out = self.cache.attend(q.cuda(), max(new), shared=shared)
        at = 0
        for b, n in enumerate(new):
            self.k[b], self.v[b] = torch.cat((self.k[b], k[at:at + n])), torch.cat((self.v[b], v[at:at + n]))
            at += n
        assert self.cache.status.tolist()[2:] == [0, 0]
        self.check(q, new, out)

    def check(self, q=None, new=None, out=None):
        c = self.cache
        lens = [len(x) for x in self.k]
        assert c.lens.tolist() == lens
        table, codes, scales = c.block_table.cpu(), c.codes.cpu(), c.scales.cpu()
        holders = [0] * self.pages
        for b, n in enumerate(lens):
            row = table[b].tolist()
            held = -(-n // P)
            assert all(p >= 0 for p in row[:held]) and all(p == -1 for p in row[held:])
            for p in row[:held]:
                holders[p] += 1
            if n:
                j = torch.arange(n)
                got = ref.gather(codes, scales, c.codebook.cpu(), table[b].long()[j // P], j % P)
                for kv, x in enumerate((self.k[b], self.v[b])):
                    code, s = ref.encode(x, c.codebook[kv].cpu())
                    want = torch.gather(c.codebook[kv].cpu().double()[None].expand(n, -1, -1), 2, code.long()) * s[..., None]
                    assert torch.equal(got[kv], want)
        free = c.free_pages[:int(c.free_count)].tolist()
        assert sorted(free + [p for p in range(self.pages) if holders[p]]) == list(range(self.pages))
        assert c.shares.tolist() == [max(0, n - 1) for n in holders]
        if out is not None:
            cu = [sum(new[:b]) for b in range(len(new) + 1)]
            want = ref.attention(q, cu, lens, table, c.codebook.cpu(), codes, scales, 1 / math.sqrt(D), True, 0)
            tol, _ = ref.attention_tolerance(*want, D, q.dtype)
            assert bool(((out.cpu().double() - want[0]).abs() <= tol).all())

    def fork(self, rows, sources, keep=None):
        self.cache.fork(i32(rows), i32(sources), keep=None if keep is None else i32(keep))
        k, v = list(self.k), list(self.v)
        for i, (r, s) in enumerate(zip(rows, sources)):
            n = len(k[s]) if keep is None else keep[i]
            self.k[r], self.v[r] = k[s][:n], v[s][:n]


def test_samples_of_a_prompt():
    s = Serving(60, 6)
    s.step([100, 0, 0, 70, 0, 0])
    s.fork([1, 2, 4], [0, 0, 3])
    s.check()
    groups = (i32([0, 3, 5]), i32([96, 64]))
    for _ in range(3):
        s.step([1, 1, 2, 1, 1, 0], shared=groups)
    s.cache.release(i32([0, 3]))
    s.k[0] = s.k[3] = s.v[0] = s.v[3] = s.k[0][:0]
    s.step([0, 5, 40, 33, 1, 9])


def test_beams():
    r = random.Random(1)
    s = Serving(80, 5)
    s.step([90] * 5)
    for _ in range(6):
        s.fork(list(range(5)), [r.randrange(5) for _ in range(5)])
        s.step([1] * 5)
    # a row taken back into what it shares, then written on
    s.cache.release(i32([0, 2]), keep=i32([50, 64]))
    for b, n in ((0, 50), (2, 64)):
        s.k[b], s.v[b] = s.k[b][:n], s.v[b][:n]
    s.check()
    s.step([3, 1, 40, 1, 1])


def test_forks_of_parts_and_compaction():
    s = Serving(64, 4)
    s.step([300, 33, 1, 64])
    s.fork([1, 2], [0, 0], keep=[128, 45])
    s.step([1, 2, 3, 4])
    s.cache.release(i32([0]))
    s.k[0] = s.v[0] = s.k[0][:0]
    s.cache.compact()
    s.check()
    used = 64 - int(s.cache.free_count)
    assert int(s.cache.block_table.max()) == used - 1
    s.step([70, 1, 1, 1])
    s.cache.compact()
    s.check()


def test_compaction_of_an_empty_and_a_full_pool():
    s = Serving(14, 2)                                               # 366 and 50 tokens: 12 + 2 pages
    s.cache.compact()
    s.check()
    s.step([13 * P - 50, 50])
    assert int(s.cache.free_count) == 0
    s.cache.compact()
    s.step([0, 14])


def test_another_cache_on_the_same_table():
    # a second layer: the copies are made there too
    s = Serving(40, 3)
    s.step([70, 0, 0])
    codes, scales = s.cache.codes.clone(), s.cache.scales.clone()
    copies = s.cache.fork(i32([1, 2]), i32([0, 0]))
    fk.fk_kv4_copy(copies, codes, scales)
    assert torch.equal(codes, s.cache.codes) and torch.equal(scales, s.cache.scales)
    moves = s.cache.release(i32([0]), keep=40)
    fk.fk_kv4_copy(moves, codes, scales)
    moves = s.cache.compact()
    fk.fk_kv4_copy(moves, codes, scales)
    assert torch.equal(codes, s.cache.codes) and torch.equal(scales, s.cache.scales)


def test_rows_and_sources():
    s = Serving(20, 4)
    s.step([40, 10, 0, 0])
    s.cache.fork([-1, 7], torch.tensor([0, 1], device="cuda"))      # the last row; none
    s.k[3], s.v[3] = s.k[0], s.v[0]
    s.check()
    s.cache.fork(i32([0]), i32([9]))                                 # a source that is none is empty
    s.k[0] = s.v[0] = s.k[0][:0]
    s.check()
    s.cache.fork([], [])
    with pytest.raises(ValueError):
        s.cache.fork([1, 2], [0])
    s.check()


@pytest.mark.parametrize("greedy", [False, True])
def test_drafts(greedy):
    # four tokens a step, some of them kept; the next step goes on behind them
    V, R = 50, 3
    s = Serving(40, R)
    s.step([30, 64, 5])
    for step in range(4):
        new = [4, 1, 0] if step % 2 else [2, 4, 3]
        T = sum(new)
        s.step(new)
        g = torch.Generator("cuda").manual_seed(step)
        p = torch.rand(T, V, device="cuda", generator=g).softmax(-1)
        q = torch.rand(T, V, device="cuda", generator=g).softmax(-1)
        tokens = p.argmax(-1).roll(1).int() if greedy else torch.multinomial(q, 1, generator=g)[:, 0].int()
        tokens[1] = 3
        u, pick = torch.rand(T, device="cuda", generator=g), torch.rand(R, device="cuda", generator=g)
        cu = s.cache.cu.tolist()
        lens = s.cache.lens.tolist()
        if greedy:
            accepted, emitted = s.cache.verify(tokens, p)
            a, e, keep = serve_ref.verify(cu, tokens.tolist(), p, None, None, None, lens)
        else:
            accepted, emitted = s.cache.verify(tokens, p, q, u, pick)
            a, e, keep = serve_ref.verify(cu, tokens.tolist(), p, q, u.tolist(), pick.tolist(), lens)
        assert accepted.tolist() == a and emitted.tolist() == [e[r] for r in range(T)]
        for b, n in enumerate(keep):
            s.k[b], s.v[b] = s.k[b][:n], s.v[b][:n]
        s.check()


def test_rotated_rows():
    # the score of two rotated rows depends on the distance of their positions alone
    s = Serving(20, 2)
    s.cache.plan(i32([5, 7]), 12)
    q, k = (torch.randn(1, h, D, generator=s.g).expand(12, h, D).contiguous().cuda() for h in (Hq, H))
    turns = fk.rope_turns(D)
    s.cache.rotate(q, k, turns)
    assert s.cache.positions.tolist() == [0, 1, 2, 3, 4, 0, 1, 2, 3, 4, 5, 6]
    x = torch.einsum("tgd,shd->tsgh", q.cpu().double(), k.cpu().double())
    # |q| |k| times a few roundings of 2^-24 a pair of products
    tol = 40 * 2.0 ** -24 * float(q.norm(dim=-1).max() * k.norm(dim=-1).max())
    for d in range(5):
        near = [x[i + d, i] for i in range(5 - d)] + [x[5 + i + d, 5 + i] for i in range(7 - d)]
        assert all(float((y - near[0]).abs().max()) < tol for y in near)


def test_a_step_captured():
    # plan, rotate, append, attend, verify and release as one graph, replayed
    R, V, new = 3, 40, 2
    caches = [fk.KV4Cache(30, P, H, D, ref.codebook(H, 0).cuda(), R, 300) for _ in range(2)]
    g = torch.Generator("cuda").manual_seed(3)
    T, turns = R * new, fk.rope_turns(D)
    n = i32([new] * R)
    data = [torch.empty(T, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H)]
    p, tokens = torch.empty(T, V, device="cuda"), i32([0] * T)
    u, pick = torch.empty(T, device="cuda"), torch.empty(R, device="cuda")

    def step(c):
        c.plan(n, T)
        q, k = data[0].clone(), data[1].clone()
        c.rotate(q, k, turns)
        c.append(k, data[2])
        out = c.attend(q, new)
        accepted, emitted = c.verify(tokens, p, None, u, pick)
        return out, accepted, emitted

    def fill(seed):
        for t in data:
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        p.copy_(torch.randn(T, V, device="cuda", generator=g).softmax(-1))
        tokens.copy_(p.argmax(-1).roll(1))
        u.copy_(torch.rand(T, device="cuda", generator=g) * 0.2)
        pick.copy_(torch.rand(R, device="cuda", generator=g))
    # the buffers of lengths change places each step: two steps are captured
    fill(0)
    for c in caches:
        step(c), step(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first, second = step(caches[0]), step(caches[0])
    for seed in range(3):
        fill(seed)
        graph.replay()
        want = step(caches[1]), step(caches[1])
        torch.cuda.synchronize()
        for a, b in zip((*first, *second), (*want[0], *want[1])):
            assert torch.equal(a, b)
        assert torch.equal(caches[0].lens, caches[1].lens) and torch.equal(caches[0].block_table, caches[1].block_table)


def test_more_rows_than_a_call_takes():
    # 70000 names of the same rows: each is shortened to the least of its lengths, once
    s = Serving(20, 4)
    s.step([100, 64, 33, 0])
    rows = torch.arange(70000, device="cuda") % 4
    keep = torch.full((70000,), 90, device="cuda")
    keep[69990:] = 40                                                # in the second call
    s.cache.release(rows, keep=keep)
    for b, n in enumerate([40, 40, 33, 0]):
        s.k[b], s.v[b] = s.k[b][:n], s.v[b][:n]
    s.check()


def test_all_of_it_on_another_stream():
    # what the calls take for themselves belongs to the stream they run on
    side = torch.cuda.Stream()
    V, out = 3000, []
    for stream in (None, side):
        g = torch.Generator("cuda").manual_seed(5)
        cache = fk.KV4Cache(60, P, H, D, ref.codebook(H, 0).cuda(), 4, 400)
        q, k, v = (torch.randn(43, h, D, device="cuda", generator=g).bfloat16() for h in (Hq, H, H))
        p = torch.rand(43, V, device="cuda", generator=g).softmax(-1)
        u, pick = torch.rand(43, device="cuda", generator=g), torch.rand(4, device="cuda", generator=g)
        n, rows, src, turns = i32([40, 1, 2, 0]), i32([1, 2, 3]), i32([0, 0, 0]), fk.rope_turns(D)
        cug, prefix, tokens = i32([0, 4]), i32([32]), p.argmax(-1).roll(1).int()
        ones, zero = i32([1, 1, 1, 1]), i32([0])                     # inputs live until the stream has run
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        if stream is not None:
            stall(stream)
        cache.plan(n, 43, stream=stream)
        cache.rotate(q, k, turns, stream=stream)
        cache.append(k, v, stream=stream)
        a = cache.attend(q, 40, stream=stream)
        b = cache.verify(tokens, p, None, u, pick, stream=stream)
        c = cache.fork(rows, src, stream=stream)
        cache.plan(ones, 4, stream=stream)
        cache.append(k[:4], v[:4], stream=stream)
        e = cache.attend(q[:4], 1, shared=(cug, prefix), stream=stream)
        cache.release(zero, stream=stream)
        f = cache.compact(stream=stream)
        assert stream is None or Bystanders([1 << 12, 1 << 16, 1 << 20]).untouched()
        torch.cuda.synchronize()
        out.append([a, *b, c, e, f, cache.lens, cache.block_table, cache.shares, cache.codes, cache.scales])
    for x, y in zip(*out):
        assert torch.equal(x, y)


def test_two_graphs_on_one_workspace():
    # forks and verification captured twice with the same workspaces, replayed in turn
    R, V = 6, 900
    s = Serving(50, R)
    s.step([70, 33, 1, 64, 0, 5])
    c = s.cache
    ws = fk.kv_fork_workspace(R, c.block_table, c.shares)
    pool = (P, c.block_table, c.lens, c.shares, c.free_pages, c.free_count)
    copies = i32([[0] * 3] * R)
    plans = [([4, 2], [0, 3], [70, 64]), ([1, 0, 5], [1, 4, 0], [20, 50, 60])]
    p = torch.rand(5, V, device="cuda").softmax(-1)
    cu, tokens, u, pick = i32([0, 2, 5]), i32([0, 3, 0, 5, 7]), torch.rand(5, device="cuda"), torch.rand(2, device="cuda")
    vws, accepted, emitted = fk.verify_workspace(cu, p), [i32([0, 0]) for _ in plans], [i32([0] * 5) for _ in plans]
    args = [(i32(a), i32(b), i32(k)) for a, b, k in plans]
    graphs = []
    for i, (a, b, k) in enumerate(args):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fk.fk_kv_fork(a, b, k, *pool, copies[:len(a)], seq=c._seq, ws=ws)
            fk.fk_kv4_copy(copies[:len(a)], c.codes, c.scales)
            fk.fk_verify(cu, tokens, p, accepted[i], emitted[i], accept=u if i else None, pick=pick if i else None, ws=vws)
    want = [serve_ref.verify([0, 2, 5], tokens.tolist(), p, None, u.tolist() if i else None, pick.tolist() if i else None, [0, 0]) for i in (0, 1)]
    for turn in range(4):
        i = turn % 2
        graphs[i].replay()
        rows, src, keep = plans[i]
        k, v = list(s.k), list(s.v)
        for r, x, n in zip(rows, src, keep):
            s.k[r], s.v[r] = k[x][:n], v[x][:n]
        s.check()
        assert accepted[i].tolist() == want[i][0] and emitted[i].tolist() == [want[i][1][r] for r in range(5)]
