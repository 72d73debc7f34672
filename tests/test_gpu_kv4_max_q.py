"""A request with more query tokens than max_q says: the tokens from max_q on
are left out, and nothing else changes."""
import math

import numpy as np
import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref

pytestmark = pytest.mark.gpu
DT = ref.DT
GUARD = 1 << 16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def attend(seq, qlen, said, Hq, H, D, dtype, extra):
    P, B = 32, len(seq)
    g = torch.Generator().manual_seed(said)
    held = [-(-s // P) for s in seq]
    table = torch.full((B, max(held) + extra), -1, dtype=torch.int32)
    used = 0
    for b, n in enumerate(held):
        table[b, :n] = torch.arange(used, used + n)
        used += n
    codes = torch.randint(0, 256, (used, H, 2, 1, 16 * D), dtype=torch.uint8, generator=g)
    scales = (1 + torch.rand(used, H, 2, P, generator=g)).to(DT[dtype])
    cb = ref.codebook(H, 1)
    cu = torch.tensor([0] + list(np.cumsum(qlen)), dtype=torch.int32)
    T, scale = int(cu[-1]), 1 / math.sqrt(D)
    q = torch.randn(T, Hq, D, generator=g).to(DT[dtype])
    out = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    dev = [t.cuda() for t in (q, cu, torch.tensor(seq, dtype=torch.int32), table, cb, codes, scales)]
    # nothing past the workspace is touched
    n = fk.kv4_attention_workspace(dev[0], dev[2], dev[5], said).numel()
    ws = torch.full((n + GUARD,), 0x5a, dtype=torch.uint8, device="cuda")
    fk.fk_kv4_attention(*dev, out, said, scale=scale, lse=lse, ws=ws[:n])
    assert bool((ws[n:] == 0x5a).all())
    o, l, *bounds = ref.attention(q, cu, seq, table, cb, codes, scales, scale, True, 0)
    tol, tol_lse = ref.attention_tolerance(o, l, *bounds, D, out.dtype)
    keep = torch.cat([torch.arange(x) < said for x in qlen])
    out, lse = out.cpu(), lse.cpu()
    assert bool(((out.double() - o).abs() <= tol)[keep].all())
    ok = keep[:, None] & torch.isfinite(l)
    assert bool(((lse.double() - l).abs() <= tol_lse)[ok].all())
    assert bool((out[~keep] == 7).all()) and bool((lse[~keep] == 7).all())


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (256, "f16")])
@pytest.mark.parametrize("extra", [0, 200])         # one launch, and shares with a join
@pytest.mark.parametrize("said,qlen", [(1, [1, 2, 1, 9, 1]), (3, [3, 40, 2, 3, 5]), (20, [7, 21, 100, 1, 20])])
def test_tokens_from_max_q_on_are_left_out(said, qlen, extra, D, dtype):
    attend([700, 300, 1500, 64, 33], qlen, said, 8, 2, D, dtype, extra)


@pytest.mark.parametrize("D,H", [(64, 110), (128, 90), (256, 32)])
def test_of_prompts_that_fill_the_card(D, H):
    attend([90], [90], 70, 12 * H, H, D, "bf16", 0)
