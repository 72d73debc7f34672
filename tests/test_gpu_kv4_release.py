"""KV4Cache.release: every page is in the list or in the table, once, whatever
rows are named; drafts are taken back and their pages used again."""
import math

import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref
from test_gpu_streams import stall

pytestmark = pytest.mark.gpu
H, Hq, D, P, PAGES, B = 2, 4, 64, 32, 30, 4


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(lens):
    cache = fk.KV4Cache(PAGES, P, H, D, ref.codebook(H, 0).cuda(), B, 320)
    cache.plan(i32(lens), sum(lens))
    return cache


def check(cache, lens):
    assert cache.lens.tolist() == lens
    held = [-(-n // P) for n in lens]
    table = cache.block_table.tolist()
    for row, n in zip(table, held):
        assert all(p >= 0 for p in row[:n]) and all(p == -1 for p in row[n:])
    left = cache.free_pages[:int(cache.free_count)].tolist()
    assert sorted(left + [p for row in table for p in row if p >= 0]) == list(range(PAGES))


@pytest.mark.parametrize("rows,gone", [
    ([1, 3], [1, 3]), ([2, 2], [2]), ([0, 3, 0, 3, 3], [0, 3]), ([-1], [3]), ([-1, 3], [3]),
    ([4], []), ([-5, 1, 400], [1]), ([], []), ([3, 1, 2, 0], [0, 1, 2, 3])])
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_rows(rows, gone, dtype):
    lens = [40, 100, 64, 33]
    cache = filled(lens)
    cache.release(torch.tensor(rows, dtype=dtype, device="cuda"))
    check(cache, [0 if b in gone else n for b, n in enumerate(lens)])


def test_a_mask_of_rows():
    cache = filled([40, 100, 64, 33])
    cache.release(torch.tensor([True, False, False, True], device="cuda"))
    check(cache, [0, 100, 64, 0])


@pytest.mark.parametrize("rows,keep,left", [
    ([1], 65, {1: 65}), ([1], 64, {1: 64}), ([1], 97, {1: 97}), ([0, 2], 33, {0: 33, 2: 33}),
    ([0, 1, 2, 3], [40, 96, 0, 500], {1: 96, 2: 0}), ([1, 1], [99, 31], {1: 31}), ([2], -3, {2: 0}), ([9], 0, {})])
def test_first_tokens_are_kept(rows, keep, left):
    lens = [40, 100, 64, 33]
    cache = filled(lens)
    cache.release(torch.tensor(rows, device="cuda"), keep=keep if isinstance(keep, int) else i32(keep))
    check(cache, [left.get(b, n) for b, n in enumerate(lens)])


def test_drafts_are_taken_back():
    g = torch.Generator().manual_seed(0)
    cache, cb = filled([0, 0, 0, 0]), ref.codebook(H, 0)
    lens, rows = [0] * B, torch.arange(B, device="cuda")
    for step in range(30):
        new = [30, 5, 1, 62] if step == 0 else [5] * B              # pages end inside the drafts
        T = sum(new)
        q, k, v = (torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, H, H))
        _, positions, cu = cache.plan(i32(new), T)
        assert positions.tolist() == [n + i for n, m in zip(lens, new) for i in range(m)]
        cache.append(k.cuda(), v.cuda())
        out = cache.attend(q.cuda(), max(new))
        seq = [a + b for a, b in zip(lens, new)]
        want = ref.attention(q, cu.cpu(), seq, cache.block_table.cpu(), cb, cache.codes.cpu(), cache.scales.cpu(),
                             1 / math.sqrt(D), True, 0)
        tol, _ = ref.attention_tolerance(*want, D, torch.bfloat16)
        assert bool(((out.cpu().double() - want[0]).abs() <= tol).all())
        taken = new if step == 0 else torch.randint(0, 6, (B,), generator=g).tolist()
        lens = [a + b for a, b in zip(lens, taken)]
        cache.release(rows, keep=i32(lens))
        check(cache, lens)
    assert cache.status.tolist()[2:] == [0, 0]


@pytest.mark.parametrize("keep,lens", [(None, [40, 0, 64, 0]), (33, [40, 33, 64, 33]), ([33, 0], [40, 33, 64, 0])])
def test_release_does_not_wait(keep, lens):
    keep = i32(keep) if isinstance(keep, list) else keep
    rows = torch.tensor([1, 3], device="cuda")
    for busy in (False, True):                       # the first call loads the kernels
        cache, done = filled([40, 100, 64, 33]), torch.cuda.Event()
        torch.cuda.synchronize()
        if busy:
            left = stall(torch.cuda.current_stream())
        done.record()
        cache.release(rows, keep=keep)
        if busy:
            assert not done.query()
            del left
    check(cache, lens)
