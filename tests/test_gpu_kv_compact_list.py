"""fk_kv_compact in place: the list's entries behind its end stay as they were."""
import pytest
import torch

import exact_lloyd_means_amd as fk
from test_gpu_kv_pages import compact, on_gpu, pool_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


@pytest.mark.parametrize("R,M,N,P", [(1, 3, 2, 32), (4, 9, 40, 32), (7, 5, 33, 64), (50, 20, 1000, 32), (300, 40, 40000, 96)])
def test_entries_behind_the_list(R, M, N, P):
    for seed in range(3):
        pool = pool_of(R, M, N, P, seed, fill=1.0)
        left = len(pool.free)
        g = on_gpu(pool)
        g["free_pages"][left:] = torch.arange(10 ** 6, 10 ** 6 + N - left, dtype=torch.int32, device="cuda")
        before = g["free_pages"].clone()
        compact(pool, g, True)
        pool.compact()
        assert int(g["free_count"]) == left and g["free_pages"][:left].tolist() == pool.free
        assert torch.equal(g["free_pages"][left:], before[left:])
