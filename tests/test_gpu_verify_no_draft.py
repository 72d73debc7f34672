"""Verification where a row has no draft (-1, or a number beyond the vocabulary):
the token is drawn from the target, of which nothing is taken away."""
import math

import pytest
import torch

import exact_lloyd_means_amd as fk
import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(cu, tokens, p, q, u, pick):
    B, T = len(cu) - 1, len(p)
    accepted, emitted = i32([-9] * B), i32([-9] * T)
    fk.fk_verify(i32(cu), i32(tokens), p, accepted, emitted, draft=q, accept=u, pick=pick)
    return accepted.tolist(), emitted.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("none", [-1, -2 ** 31, "V", 2 ** 31 - 1])
@pytest.mark.parametrize("V", [1, 7, 1031, 20011])
@pytest.mark.parametrize("drafted", [True, False])
def test_nothing_is_taken_away(V, none, dtype, drafted):
    # what a request of that row alone samples, whose token is drawn from p
    g = torch.Generator("cuda").manual_seed(V)
    n, bad = 12, V if none == "V" else none
    p, q = (torch.randn(2 * n, V, device="cuda", generator=g).softmax(-1).to(dtype) for _ in range(2))
    pick = torch.rand(n, device="cuda", generator=g)
    accepted, emitted = run([2 * b for b in range(n + 1)], [bad] * (2 * n), p, q if drafted else None, torch.zeros(2 * n, device="cuda"), pick)
    _, want, _ = ref.verify(list(range(n + 1)), [0] * n, p[::2], None, [0.0] * n, pick.tolist(), [0] * n)
    assert accepted == [0] * n
    assert emitted == [x for b in range(n) for x in (want[b], -1)]


def test_drafts_before_it_count():
    # a draft that is kept, then none; and none behind one that is refused changes nothing
    V = 5
    p = torch.tensor([[0.1, 0.6, 0.1, 0.1, 0.1], [0.0, 0.0, 0.0, 0.5, 0.5], [0.2] * 5] * 2, device="cuda")
    q = torch.tensor([[0.1, 0.6, 0.1, 0.1, 0.1], [0.0, 0.0, 0.0, 0.9, 0.1], [0.2] * 5] * 2, device="cuda")
    u = torch.tensor([0.5, 0.5, 0.5, 1.0 - 2.0 ** -24, 0.0, 0.0], device="cuda")
    p[3, 1] = 0.1                                     # 0.999 0.6 < 0.1 is not so
    accepted, emitted = run([0, 3, 6], [0, 1, -1, 0, 1, -1], p, q, u, torch.tensor([0.25, 0.0], device="cuda"))
    # p of row 1 at a quarter of its sum: 3 (p - q would leave 4 alone); of row 3 nothing but zeros is left, so p: 0
    assert accepted == [1, 0] and emitted == [1, 3, -1, 0, -1, -1]


def test_distribution():
    # half of the requests have a draft: the first token is distributed as the target says for all
    V, B = 6, 20000
    g = torch.Generator("cuda").manual_seed(0)
    p = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1], device="cuda").expand(2 * B, V)
    q = torch.tensor([0.3, 0.1, 0.3, 0.1, 0.1, 0.1], device="cuda").expand(2 * B, V)
    d = torch.multinomial(q[0], 2 * B, True, generator=g).int()
    d[1::4] = -1
    cu = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda")
    accepted, emitted = i32([0] * B), i32([0] * (2 * B))
    fk.fk_verify(cu, d, p, accepted, emitted, draft=q, accept=torch.rand(2 * B, device="cuda", generator=g),
                 pick=torch.rand(B, device="cuda", generator=g))
    for first in (0, 2):                              # without a draft, with one
        got = torch.bincount(emitted[first::4].long(), minlength=V).double() / (B // 2)
        # five standard deviations of a share: 5 sqrt(0.25 / (B / 2))
        assert float((got - p[0].double()).abs().max()) < 5 * math.sqrt(0.5 / B)
