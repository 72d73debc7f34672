"""Pages of the cache on the GPU: forked, returned, copied and compacted, against
a pool of lists."""
import random

import pytest
import torch

import exact_lloyd_means_amd as fk
import serve_ref as ref
from test_gpu_streams import Bystanders, stall

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool_of(R, M, N, P, seed, fill=0.7):
    r = random.Random(seed)
    ids = list(range(N))
    r.shuffle(ids)
    lens, table = [0] * R, [[-1] * M for _ in range(R)]
    for b in range(R):
        n = r.choice([0, 1, P - 1, P, P + 1, r.randrange(M * P + 1), r.randrange(M * P + 1)])
        k = -(-n // P)
        if k <= len(ids) - int((1 - fill) * N):
            table[b][:k] = [ids.pop() for _ in range(k)]
            lens[b] = n
    return ref.Pool(table, lens, ids, N, P, seq=[n + 3 for n in lens])


def on_gpu(pool):
    N = pool.pages
    return dict(block_table=i32(pool.table), lens=i32(pool.lens), shares=i32(pool.shares()),
                free_pages=i32(pool.free + [-7] * (N - len(pool.free))), free_count=i32([len(pool.free)]))


def same(pool, g):
    assert g["block_table"].tolist() == pool.table
    assert g["lens"].tolist() == pool.lens
    assert g["shares"].tolist() == pool.shares()
    assert int(g["free_count"]) == len(pool.free)
    assert g["free_pages"].tolist()[:len(pool.free)] == pool.free
    n = pool.holders()
    assert sorted(pool.free + [p for p in range(pool.pages) if n[p]]) == list(range(pool.pages))


def fork(pool, g, rows, sources, keep, seq=None, ws=None, stream=None):
    copies = i32([[-9] * 3] * len(rows))
    fk.fk_kv_fork(i32(rows), None if sources is None else i32(sources), i32(keep), pool.P, copies=copies, seq=seq, ws=ws, stream=stream, **g)
    torch.cuda.synchronize()
    return copies.tolist()


@pytest.mark.parametrize("n", [1, 3, 64, 65, 300])
@pytest.mark.parametrize("P", [32, 96])
def test_forks_follow_each_other(n, P):
    R, M = max(4, n // 2), 9
    for seed in range(4):
        r = random.Random(seed * n)
        pool = pool_of(R, M, R * M // 2 + 5, P, seed)
        g = on_gpu(pool)
        seq = i32(pool.seq)
        for _ in range(6):
            rows = [r.randrange(-1, R + 1) for _ in range(n)] if r.random() < 0.5 else (r.sample(range(R), R) * 2)[:n]
            sources = [r.randrange(-1, R + 1) for _ in rows] if r.random() < 0.7 else None
            keep = [r.choice([-1, 0, 1, P, P + 1, 3 * P, r.randrange(M * P), 2 ** 31 - 1]) for _ in rows]
            want = pool.fork(rows, sources, keep)
            assert fork(pool, g, rows, sources, keep, seq=seq) == want
            same(pool, g)
            assert seq.tolist() == pool.seq


def test_rows_longer_than_a_wave():
    R, M, P = 5, 300, 32
    pool = pool_of(R, M, 900, P, 3, fill=1.0)
    g = on_gpu(pool)
    for rows, sources, keep in (([1, 2, 3], [0, 0, 4], [9600] * 3), ([0, 1], None, [4000, 77]), ([2, 4, 0], [4, 2, 1], [5000, 9000, 64])):
        want = pool.fork(rows, sources, keep)
        assert fork(pool, g, rows, sources, keep) == want
        same(pool, g)


def test_swapped_rows_copy_nothing():
    pool = ref.Pool([[0, 1], [2, 3]], [40, 50], [5, 4], 6, 32)
    g = on_gpu(pool)
    assert fork(pool, g, [0, 1], [1, 0], [64, 64]) == [[-1, -1, 0]] * 2
    pool.fork([0, 1], [1, 0], [64, 64])
    same(pool, g)
    assert pool.table == [[2, 3], [0, 1]]


def test_no_page_for_a_copy():
    # three continuations of a row with a partly filled page, one page in the list: the later ones end with whole pages
    pool = ref.Pool([[0, 1]] + [[-1, -1]] * 3, [50, 0, 0, 0], [2], 3, 32)
    g = on_gpu(pool)
    copies = fork(pool, g, [1, 2, 3], [0, 0, 0], [64] * 3)
    assert copies == [[1, 2, 18], [-1, -1, 0], [-1, -1, 0]] == pool.fork([1, 2, 3], [0, 0, 0], [64] * 3)
    same(pool, g)
    assert pool.lens == [50, 50, 32, 32]


def test_on_another_stream():
    pool = pool_of(200, 6, 700, 32, 5)
    g = on_gpu(pool)
    rows, sources, keep = i32(list(range(100))), i32([100 + i % 50 for i in range(100)]), i32([150] * 100)
    copies, side = i32([[-9] * 3] * 100), torch.cuda.Stream()
    size = fk.kv_fork_workspace(100, g["block_table"], g["shares"]).numel()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stall(side)
    fk.fk_kv_fork(rows, sources, keep, 32, copies=copies, stream=side, **g)
    assert Bystanders([size]).untouched()
    assert copies.tolist() == pool.fork(rows.tolist(), sources.tolist(), keep.tolist())
    same(pool, g)


@pytest.mark.parametrize("n", [5, 100])
def test_captured(n):
    # beams that follow each other: every replay sees what the one before left
    R, P = n, 32
    pool = pool_of(R, 5, 4 * R, P, 9)
    g = on_gpu(pool)
    rows, sources, keep, copies = i32([0] * n), i32([0] * n), i32([0] * n), i32([[0] * 3] * n)
    ws = fk.kv_fork_workspace(n, g["block_table"], g["shares"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fk.fk_kv_fork(rows, sources, keep, P, copies=copies, ws=ws, **g)
    for seed in range(4):
        r = random.Random(seed)
        a, b, c = (r.sample(range(R), n), [r.randrange(R) for _ in range(n)], [r.randrange(5 * P) for _ in range(n)])
        for t, x in ((rows, a), (sources, b), (keep, c)):
            t.copy_(i32(x))
        ws.fill_(77)
        graph.replay()
        assert copies.tolist() == pool.fork(a, b, c)
        same(pool, g)


# ---- copies --------------------------------------------------------------------------

def storage(pages, H, D, P, dtype, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (pages, H, 2, P // 32, 16 * D), dtype=torch.uint8, device="cuda", generator=g)
    return codes, torch.randn(pages, H, 2, P, device="cuda", generator=g).to(dtype)


@pytest.mark.parametrize("H,D,P,dtype", [(1, 64, 32, torch.float16), (3, 128, 96, torch.bfloat16), (8, 128, 64, torch.bfloat16),
                                         (2, 256, 1024, torch.float16), (17, 64, 224, torch.bfloat16)])
def test_copies(H, D, P, dtype):
    pages = 12
    codes, scales = storage(pages, H, D, P, dtype)
    scales[3] = float("nan")
    want_c, want_s = codes.clone(), scales.clone()
    copies = [[0, 5, 1], [0, 6, 32], [1, 7, P], [3, 8, P - 31], [2, 9, 10 ** 9], [-1, -1, 0], [1, -1, 5], [pages, 10, 5], [1, pages, 5], [1, 10, 0],
              [1, 10, -4], [-5, 10, 7]]
    for s, d, n in copies:
        if 0 <= s < pages and 0 <= d < pages and n > 0:
            b = min(-(-n // 32), P // 32)
            want_c[d, :, :, :b], want_s[d, :, :, :32 * b] = codes[s, :, :, :b], scales[s, :, :, :32 * b]
    fk.fk_kv4_copy(i32(copies), codes, scales)
    torch.cuda.synchronize()
    assert torch.equal(codes, want_c) and torch.equal(scales.view(torch.int16), want_s.view(torch.int16))


def test_copies_beyond_32_bits():
    # more than 2^32 bytes of codes
    pages, H, D, P = 66000, 8, 128, 64
    codes = torch.zeros(pages, H, 2, 2, 16 * D, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, H, 2, P, dtype=torch.float16, device="cuda")
    codes[pages - 1], scales[pages - 1] = 7, 3
    fk.fk_kv4_copy(i32([[pages - 1, 0, P], [pages - 1, pages - 2, P]]), codes, scales)
    assert bool((codes[[0, pages - 2]] == 7).all()) and bool((scales[[0, pages - 2]] == 3).all())
    assert not bool(codes[1:pages - 2].any()) and not bool(scales[1:pages - 2].any())


# ---- compaction -------------------------------------------------------------------------

def compact(pool, g, in_place, more=0, stream=None):
    N = pool.pages
    new = [g["block_table"], g["shares"], g["free_pages"], g["free_count"]]
    if not in_place:
        new = [torch.full_like(t, -9) for t in new]
    moves = i32([[-9] * 3] * (N // 2 + more)).view(-1, 3)
    fk.fk_kv_compact(pool.P, g["block_table"], g["lens"], g["shares"], g["free_pages"], g["free_count"], *new, moves, stream=stream)
    torch.cuda.synchronize()
    return new, moves.tolist()


@pytest.mark.parametrize("R,M,N,P", [(1, 1, 1, 32), (1, 3, 2, 32), (4, 9, 40, 32), (7, 5, 33, 64), (50, 20, 1000, 32), (300, 40, 40000, 96)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compaction(R, M, N, P, in_place):
    for seed in range(3):
        pool = pool_of(R, M, N, P, seed, fill=1.0)
        if R > 3:                                     # rows that share pages
            pool.fork([0, 1], [2, 2], [10 ** 6] * 2)
        g = on_gpu(pool)
        (table, shares, free, left), moves = compact(pool, g, in_place, more=seed)
        want = pool.compact()
        assert moves == want + [[-1, -1, 0]] * (N // 2 + seed - len(want))
        assert table.tolist() == pool.table and shares.tolist() == pool.shares()
        assert int(left) == len(pool.free) and free.tolist()[:len(pool.free)] == pool.free
        assert free.tolist()[len(pool.free):] == ([-9] * (N - len(pool.free)) if not in_place else free.tolist()[len(pool.free):])


def test_compaction_of_the_largest_pool():
    N, P = 1 << 20, 32
    used = torch.arange(N - 64, N, dtype=torch.int32, device="cuda")
    table, lens = used.view(1, 64).clone(), i32([64 * P])
    free = torch.cat((torch.arange(N - 64, dtype=torch.int32, device="cuda"), i32([-1] * 64)))
    g = dict(block_table=table, lens=lens, shares=torch.zeros(N, dtype=torch.int32, device="cuda"), free_pages=free, free_count=i32([N - 64]))
    g["shares"][N - 1] = 5
    moves = torch.empty(N // 2, 3, dtype=torch.int32, device="cuda")
    fk.fk_kv_compact(P, **g, new_table=table, new_shares=g["shares"], new_free=free, free_left=g["free_count"], moves=moves)
    assert table.tolist() == [list(range(64))] and int(g["free_count"]) == N - 64
    assert torch.equal(free[:N - 64], torch.arange(N - 1, 63, -1, dtype=torch.int32, device="cuda"))
    assert moves[:65].tolist() == [[N - 64 + i, i, P] for i in range(64)] + [[-1, -1, 0]]
    assert int(g["shares"][63]) == 5 and int(g["shares"].sum()) == 5
