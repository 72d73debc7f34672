"""Forks and returns of thousands of rows: the same as of few, in time that follows
their number."""
import random

import pytest
import torch

import exact_lloyd_means_amd as fk
import serve_ref as ref
from test_gpu_kv_pages import fork, i32, on_gpu, pool_of, same
from test_gpu_streams import Bystanders, stall

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


@pytest.mark.parametrize("n,R", [(1023, 700), (1024, 700), (1025, 40), (5000, 4000), (3001, 3001)])
def test_as_a_pool_of_lists(n, R):
    M, P = 4, 32
    r = random.Random(n)
    pool = pool_of(R, M, R * 2 + 40, P, n)
    g = on_gpu(pool)
    seq = i32(pool.seq)
    for turn in range(3):
        rows = r.sample(range(R), R) if n == R else [r.randrange(-1, R + 1) for _ in range(n)]
        sources = None if turn == 1 else [r.randrange(-1, R + 1) for _ in rows]
        keep = [r.choice([-1, 0, 1, P, P + 1, r.randrange(M * P), 2 ** 31 - 1]) for _ in rows]
        want = pool.fork(rows, sources, keep)
        assert fork(pool, g, rows, sources, keep, seq=seq) == want
        same(pool, g)
        assert seq.tolist() == pool.seq


def test_no_pages_for_the_last_copies():
    # 3000 continuations of one partly filled page, 2500 pages in the list
    R, P = 3001, 32
    pool = ref.Pool([[0, 1]] + [[-1, -1]] * 3000, [50] + [0] * 3000, list(range(2, 2502)), 2502, P)
    g = on_gpu(pool)
    rows = list(range(1, R))
    want = [[1, 2 + i, 18] if i < 2500 else [-1, -1, 0] for i in range(3000)]
    assert fork(pool, g, rows, [0] * 3000, [64] * 3000) == want == pool.fork(rows, [0] * 3000, [64] * 3000)
    same(pool, g)


def test_one_row_named_by_all():
    n, P = 65536, 32
    pool = pool_of(3, 5, 20, P, 1)
    pool.table[1], pool.lens[1] = [pool.free.pop() for _ in range(5)], 5 * P
    g = on_gpu(pool)
    keep = i32([100] * n)
    keep[40000] = 33
    copies = torch.empty(n, 3, dtype=torch.int32, device="cuda")
    fk.fk_kv_fork(i32([1] * n), None, keep, P, copies=copies, **g)
    assert pool.fork([1], None, [33]) == [[-1, -1, 0]] and bool((copies == i32([-1, -1, 0])).all())
    same(pool, g)


def test_workspace_of_more_pairs():
    # a workspace for more pairs does for fewer, whatever it holds; on a stream of its own
    n, P = 2500, 32
    pool = pool_of(n, 3, 2 * n, P, 7)
    g = on_gpu(pool)
    for m in (n, 100, 3, 2100):
        ws = fk.kv_fork_workspace(n, g["block_table"], g["shares"])
        ws.fill_(255)
        assert ws.numel() >= fk.kv_fork_workspace(m, g["block_table"], g["shares"]).numel()
        r = random.Random(m)
        rows, sources, keep = (r.sample(range(n), m), [r.randrange(n) for _ in range(m)], [r.randrange(3 * P) for _ in range(m)])
        assert fork(pool, g, rows, sources, keep, ws=ws) == pool.fork(rows, sources, keep)
        same(pool, g)
    rows, sources, keep = i32(list(range(n))), i32(list(range(n))[::-1]), i32([40] * n)
    copies, side = i32([[-9] * 3] * n), torch.cuda.Stream()
    size = fk.kv_fork_workspace(n, g["block_table"], g["shares"]).numel()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stall(side)
    fk.fk_kv_fork(rows, sources, keep, P, copies=copies, stream=side, **g)
    assert Bystanders([size]).untouched()
    assert copies.tolist() == pool.fork(rows.tolist(), sources.tolist(), keep.tolist())
    same(pool, g)


def test_captured():
    n, P = 2100, 32
    pool = pool_of(n, 3, 2 * n, P, 9)
    g = on_gpu(pool)
    rows, sources, keep, copies = i32([0] * n), i32([0] * n), i32([0] * n), i32([[0] * 3] * n)
    ws = fk.kv_fork_workspace(n, g["block_table"], g["shares"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fk.fk_kv_fork(rows, sources, keep, P, copies=copies, ws=ws, **g)
    for seed in range(3):
        r = random.Random(seed)
        a, b, c = r.sample(range(n), n), [r.randrange(n) for _ in range(n)], [r.randrange(3 * P) for _ in range(n)]
        for t, x in ((rows, a), (sources, b), (keep, c)):
            t.copy_(i32(x))
        ws.fill_(77)
        graph.replay()
        assert copies.tolist() == pool.fork(a, b, c)
        same(pool, g)


def test_time_follows_their_number():
    # four times the rows, each with a page to give up: sixteen times the time were every
    # pair to read all pairs, about four at most where it does not
    def time(R):
        table = torch.arange(2 * R, dtype=torch.int32, device="cuda").view(R, 2)
        lens, shares = torch.full((R,), 64, dtype=torch.int32, device="cuda"), torch.zeros(2 * R, dtype=torch.int32, device="cuda")
        free, count = torch.empty(2 * R, dtype=torch.int32, device="cuda"), i32([0])
        rows, keep = torch.arange(R, dtype=torch.int32, device="cuda"), torch.full((R,), 32, dtype=torch.int32, device="cuda")
        copies = torch.empty(R, 3, dtype=torch.int32, device="cuda")
        ws, least = fk.kv_fork_workspace(R, table, shares), 1e9
        for _ in range(6):
            t, n, c = table.clone(), lens.clone(), count.clone()
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            fk.fk_kv_fork(rows, None, keep, 32, t, n, shares, free, c, copies, ws=ws)
            end.record()
            torch.cuda.synchronize()
            assert int(c) == R and torch.equal(free[:R], table[:, 1])
            least = min(least, start.elapsed_time(end))
        return least
    few, many = time(16384), time(65536)
    print(f"16384 rows {1e3 * few:.0f} us, 65536 rows {1e3 * many:.0f} us")
    assert many < 8 * few
