"""KV4Cache.release: every page is in the list or in the table, once, whatever
rows are named."""
import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref

pytestmark = pytest.mark.gpu
H, D, P, PAGES, B = 2, 64, 32, 30, 4


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
