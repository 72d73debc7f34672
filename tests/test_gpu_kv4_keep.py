"""KV4Cache.fork and release with lengths that 32 bits do not hold: they are all
of a row."""
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


@pytest.mark.parametrize("much", [2 ** 31, 2 ** 32, 2 ** 40, 2 ** 63 - 1])
@pytest.mark.parametrize("as_tensor", [True, False])
def test_more_than_32_bits(much, as_tensor):
    cache = filled([40, 100, 0, 33])
    left = int(cache.free_count)
    keep = torch.full((2,), much, device="cuda") if as_tensor else much
    cache.release(torch.tensor([0, 1], device="cuda"), keep=keep)
    assert cache.lens.tolist() == [40, 100, 0, 33] and int(cache.free_count) == left
    cache.fork(torch.tensor([2, 3], device="cuda"), torch.tensor([0, 1], device="cuda"), keep=keep)
    assert cache.lens.tolist() == [40, 100, 40, 100]
    # row 3's two pages came back, the two partly filled tails of 40 and 100 tokens were copied
    assert int(cache.free_count) == left + 2 - 2
