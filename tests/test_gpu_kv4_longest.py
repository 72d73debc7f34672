"""Attention over as many cached positions as one call takes, 2^36 less a few:
block counts near 2^31 must not wrap where they are cut into shares."""
import math

import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def test_the_most_blocks_of_a_call():
    # 32 requests of 2^31 - 1024 tokens each, every page of them the same one
    B, D, P, M = 32, 64, 1024, 2 ** 21 - 1
    g = torch.Generator().manual_seed(0)
    codes = torch.randint(0, 256, (1, 1, 2, P // 32, 16 * D), dtype=torch.uint8, generator=g)
    scales = (1 + torch.rand(1, 1, 2, P, generator=g)).half()
    cb, q = ref.codebook(1, 0), torch.randn(B, 1, D, generator=g).half()
    table = torch.zeros(B, M, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros(B, 1, D, dtype=torch.float16, device="cuda"), torch.zeros(B, 1, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fk.fk_kv4_attention(q.cuda(), i32(list(range(B + 1))), i32([M * P] * B), table, cb.cuda(), codes.cuda(),
                        scales.cuda(), out, 1, lse=lse)
    torch.cuda.synchronize()
    one = torch.zeros(B, 1, dtype=torch.int32)
    o, l, pv, dot, _ = ref.attention(q, torch.arange(B + 1), [P] * B, one, cb, codes, scales, 1 / math.sqrt(D), True, 0)
    # a wave adds 2^19 blocks one after another in fp32: 2^19 * 2^-24 of the sums at worst
    assert bool(((out.cpu().double() - o).abs() <= 2.0 ** -4 * pv + 2.0 ** -11).all())
    assert bool(((lse.cpu().double() - l - math.log(M)).abs() <= 2.0 ** -4).all())
