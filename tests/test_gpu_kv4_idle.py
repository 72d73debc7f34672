"""A step of a serving loop in which no request has a token."""
import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def test_a_step_without_tokens():
    H, D, B = 2, 64, 3
    cache = fk.KV4Cache(8, 32, H, D, ref.codebook(H, 0).cuda(), B, 128)
    for new in ([0, 0, 0], [3, 0, 1], [0, 0, 0]):
        T = sum(new)
        slots, positions, cu = cache.plan(torch.tensor(new, dtype=torch.int32, device="cuda"), T)
        rows = torch.ones(T, H, D, dtype=torch.bfloat16, device="cuda")
        cache.append(rows, rows)
        out = cache.attend(torch.ones(T, 4, D, dtype=torch.bfloat16, device="cuda"), max(new))
        assert out.shape == (T, 4, D) and slots.shape == positions.shape == (T,)
        assert cu.tolist() == [0, new[0], new[0] + new[1], T]
    assert cache.lens.tolist() == [3, 0, 1] and int(cache.free_count) == 6
    # rows for a plan that has none are still refused
    cache.plan(torch.zeros(B, dtype=torch.int32, device="cuda"), 0)
    with pytest.raises(ValueError, match="k must have shape"):
        cache.append(rows[:0].new_ones(2, H, D), rows[:0].new_ones(2, H, D))
