"""Rotary positions on the GPU against their 64-bit definition."""
import math
import random

import pytest
import torch

import exact_lloyd_means_amd as fk
import serve_ref as ref

pytestmark = pytest.mark.gpu
FAR = [0, 1, 2, 4095, 65536, 131071, 1000003, (1 << 31) - 1]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def positions(T, seed):
    r = random.Random(seed)
    return [r.choice(FAR + [-1, r.randrange(5000), r.randrange(1 << 20)]) for _ in range(T)]


def check(got, x, pos, w, interleaved, inverse, factor):
    want = ref.rope(x, pos, w, interleaved, inverse, factor)
    tol = ref.rope_tolerance(x, want, w, pos, interleaved, factor, x.dtype)
    off = (got.double().cpu() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,R", [(1, 1, 1, 2, 2), (7, 4, 2, 128, 128), (33, 3, 1, 64, 32), (5, 8, 8, 80, 80), (9, 2, 1, 80, 20),
                                        (2, 6, 3, 256, 254), (3, 40, 8, 96, 64), (4, 2, 2, 1024, 1024), (65, 1, 1, 6, 4)])
def test_matches_definition(T, Hq, H, D, R, interleaved, dtype):
    g = torch.Generator("cuda").manual_seed(T * D + R)
    q, k = (torch.randn(T, h, D, device="cuda", generator=g).to(dtype) for h in (Hq, H))
    pos = positions(T, T + R)
    turns, w = fk.rope_turns(R), ref.frequencies(R)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    qo, ko = torch.full_like(q, 99), torch.full_like(k, 99)
    for inverse, factor in ((False, 1.0), (True, 1.25)):
        fk.fk_rope(q, k, p, turns, qo, ko, interleaved=interleaved, inverse=inverse, factor=factor)
        check(qo, q, pos, w, interleaved, inverse, factor)
        check(ko, k, pos, w, interleaved, inverse, factor)
    # in place, and queries alone
    x, y = q.clone(), k.clone()
    fk.fk_rope(x, y, p, turns, interleaved=interleaved, inverse=True, factor=1.25)
    assert torch.equal(x, qo) and torch.equal(y, ko)
    alone = torch.empty_like(q)
    fk.fk_rope(q, None, p, turns, alone, interleaved=interleaved, inverse=True, factor=1.25)
    assert torch.equal(alone, qo)


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("D", [64, 72])
def test_slices_of_a_projection(D, offset):
    # rows that start anywhere, in place within the projection; what lies between stays
    T, Hq, H = 11, 4, 2
    g = torch.Generator("cuda").manual_seed(D)
    buffer = torch.randn(T * ((Hq + 2 * H) * D + 3 * offset) + offset, device="cuda", generator=g).bfloat16()
    whole = buffer[offset:].view(T, -1)
    before = buffer.clone()
    q, k = whole[:, :Hq * D].unflatten(1, (Hq, D)), whole[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
    x, y = q.clone(), k.clone()
    pos = positions(T, 3)
    fk.fk_rope(q, k, torch.tensor(pos, dtype=torch.int32, device="cuda"), fk.rope_turns(D))
    check(q, x, pos, ref.frequencies(D), False, False, 1.0)
    check(k, y, pos, ref.frequencies(D), False, False, 1.0)
    q.copy_(x)
    k.copy_(y)
    assert torch.equal(buffer, before)


@pytest.mark.parametrize("kw", [dict(base=500000.0), dict(stretch=4.0), dict(stretch=32.0, trained=4096),
                                dict(stretch=8.0, trained=8192, slow=1.0, fast=4.0, base=500000.0), dict(base=1.0)])
def test_stretched_contexts(kw):
    R, T = 128, 16
    w = ref.frequencies(R, **kw)
    x = torch.randn(T, 2, R, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    pos = positions(T, 5)
    y = torch.empty_like(x)
    fk.fk_rope(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), fk.rope_turns(R, **kw), y)
    check(y, x, pos, w, False, False, 1.0)


def test_gradient():
    # the map is linear: <g, f(x)> = <f'(g), x>, and differences give it exactly up to rounding
    T, H, D, R = 5, 3, 64, 48
    g = torch.Generator("cuda").manual_seed(2)
    x, dy, e = (torch.randn(T, H, D, device="cuda", generator=g) for _ in range(3))
    pos = torch.tensor([0, 3, 1 << 20, -1, 77], dtype=torch.int32, device="cuda")
    turns = fk.rope_turns(R)

    def f(v, inverse=False):
        out = torch.empty_like(v)
        fk.fk_rope(v, None, pos, turns, out, inverse=inverse, factor=1.5)
        return out.double()
    dx = f(dy, True)
    # each value is off by at most 10 2^-24 of 1.5 (|a| + |b|) and its own rounding
    size = T * H * D * (1.5 * 2 * 10 + 2) * 2.0 ** -24 * 25
    assert abs(float((f(x) * dy).sum() - (dx * x).sum())) < size
    difference = (f((x + e).float()) - f((x - e).float())) / 2
    assert abs(float((difference * dy).sum() - (dx * e).sum())) < 4 * size


def test_large_and_many():
    # rows beyond 2^31 elements, and a second row of workgroups
    T, H, D = 70000, 250, 128
    x = torch.zeros(T, H, D, dtype=torch.float16, device="cuda")
    x[-1] = 1
    x[0] = 1
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-1] = 12345
    fk.fk_rope(x, None, pos, fk.rope_turns(D))
    check(x[-1:], torch.ones(1, H, D, dtype=torch.float16), [12345], ref.frequencies(D), False, False, 1.0)
    assert bool((x[0] == 1).all()) and not bool(x[1:-1].any())


def test_not_finite():
    x = torch.zeros(1, 1, 8, device="cuda")
    x[0, 0, 1], x[0, 0, 2] = math.inf, math.nan
    y = torch.empty_like(x)
    fk.fk_rope(x, None, torch.tensor([3], dtype=torch.int32, device="cuda"), fk.rope_turns(4), y)
    # pair (1, 3): infinite; pair (0, 2): NaN; the rest is copied
    assert y[0, 0].isfinite().tolist() == [False, False, False, False, True, True, True, True]


def test_captured():
    T, H, D = 33, 4, 128
    x = torch.randn(T, H, D, device="cuda").bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    turns, y = fk.rope_turns(D), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fk.fk_rope(x, None, pos, turns, y)
    for shift in range(3):
        pos += 1000 * shift
        graph.replay()
        want = torch.empty_like(x)
        fk.fk_rope(x, None, pos, turns, want)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_most_tokens_of_wide_rows():
    # 2^24 tokens of rows that take a workgroup each
    T, D, R = 1 << 24, 516, 514
    x = torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, (1 << 23) - 1, 1 << 23, T - 2, T - 1]
    rows = torch.randn(len(at), 1, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    x[at] = rows.cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    fk.fk_rope(x, None, pos, fk.rope_turns(R))
    check(x[at], rows, at, ref.frequencies(R), False, False, 1.0)
    assert not bool(x[5:100].any()) and not bool(x[-100:-2].any())
