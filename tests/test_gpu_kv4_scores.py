"""Attention over the 4-bit cache with scores of any size that fp32 holds:
what counts is their difference."""
import math

import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref

pytestmark = pytest.mark.gpu
P, H, Hq = 32, 1, 4
# one launch, shares with a join; one row tile and several
FORMS = [(40, 1, 0), (700, 1, 0), (700, 1, 200), (300, 20, 0), (300, 20, 200)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def attend(S, n, extra, D, ks, q, seed=0):
    """One request whose tokens all have k codes 0, k scales ks (S), v scales
    around one, and queries q in every dimension."""
    g = torch.Generator().manual_seed(seed)
    held = -(-S // P)
    codes = torch.randint(0, 256, (held, H, 2, 1, 16 * D), dtype=torch.uint8, generator=g)
    codes[:, :, 0] = 0
    scales = (1 + torch.rand(held, H, 2, P, generator=g)).bfloat16()
    at = torch.arange(S)
    scales[at // P, :, 0, at % P] = ks.bfloat16()[:, None]
    table = torch.full((1, held + extra), -1, dtype=torch.int32)
    table[0, :held] = torch.arange(held)
    cb = ref.codebook(H, 3)
    qs = torch.full((n, Hq, D), q).bfloat16()
    out = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, Hq), 7.0, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    scale = 1 / math.sqrt(D)
    fk.fk_kv4_attention(qs.cuda(), i32(0, n), i32(S), table.cuda(), cb.cuda(), codes.cuda(), scales.cuda(), out, n,
                        scale=scale, causal=False, lse=lse)
    k, v = ref.gather(codes, scales, cb, at // P, at % P)[:, :, 0]
    s = k @ qs[0, 0].double() * scale
    return out.cpu().double(), lse.cpu().double(), s, v


@pytest.mark.parametrize("S,n,extra", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("e", [-60, 0, 12, 26, 60, 112])
@pytest.mark.parametrize("sign", [1, -1])
def test_equal_scores(S, n, extra, D, e, sign):
    # codes 0 are the lowest level, about -1: scores of about sign * D/8 * 2^e
    out, lse, s, v = attend(S, n, extra, D, torch.full((S,), 2.0 ** (e // 2)), -sign * 2.0 ** (e - e // 2))
    want = v.mean(0)
    # weights are equal, so only bf16's rounding and that of the weights count
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -10 * v.abs().mean(0)
    assert bool(((out - want).abs() <= tol).all())
    assert bool(((lse - (s[0] + math.log(S))).abs() <= 2.0 ** -16 * (s[0].abs() + 16)).all())


@pytest.mark.parametrize("S,n,extra", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("e", [26, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_apart(S, n, extra, D, e, sign):
    # three tokens share the largest score, the others lie far below
    ks = torch.full((S,), 2.0 ** (e // 2) * (1.0 if sign > 0 else 4.0))
    best = torch.tensor([3, S // 2, S - 1])
    ks[best] = 2.0 ** (e // 2) * 2
    out, lse, s, v = attend(S, n, extra, D, ks, -sign * 2.0 ** (e - e // 2))
    want = v[best].mean(0)
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -10 * v[best].abs().mean(0)
    assert bool(((out - want).abs() <= tol).all())
    top = s.max()
    assert bool(((lse - (top + math.log(3))).abs() <= 2.0 ** -16 * top.abs()).all())
