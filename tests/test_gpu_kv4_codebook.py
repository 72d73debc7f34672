"""learn_codebook: samples with values that are not finite."""
import math

import pytest
import torch

import exact_lloyd_means_amd as fk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_rows_that_are_not_finite_count_as_zeros(bad):
    g = torch.Generator("cuda").manual_seed(0)
    k, v = (torch.randn(400, 3, 64, device="cuda", generator=g).bfloat16() for _ in range(2))
    k[7, 1, 5] = v[11, 2, 60] = bad
    cb = fk.learn_codebook(k, v, iters=6)
    assert bool(torch.isfinite(cb).all()) and bool((cb.diff(dim=-1) >= 0).all())
    k[7, 1], v[11, 2] = 0, 0
    assert torch.equal(cb, fk.learn_codebook(k, v, iters=6))
