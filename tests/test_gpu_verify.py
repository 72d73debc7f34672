"""Verification of drafts on the GPU against exact integers."""
import math

import pytest
import torch

import exact_lloyd_means_amd as fk
import serve_ref as ref
from test_gpu_streams import Bystanders, stall

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(cu, tokens, p, q=None, u=None, pick=None, seq=None, stream=None, more=0):
    """Runs it, compares everything with the reference; rows of no request stay as they were."""
    B, T = len(cu) - 1, len(p)
    accepted, emitted, keep = i32([-9] * B), i32([-9] * T), i32([-9] * B)
    seq = [100 + b for b in range(B)] if seq is None else seq
    fk.fk_verify(i32(cu), i32(tokens), p, accepted, emitted, draft=q, accept=u, pick=pick, seq_lens=i32(seq), keep=keep, stream=stream)
    torch.cuda.synchronize()
    a, e, k = ref.verify(cu, tokens, p, q, None if u is None else u.tolist(), None if pick is None else pick.tolist(), seq)
    assert accepted.tolist() == a
    assert emitted.tolist() == [e.get(r, -9) for r in range(T)]
    assert keep.tolist() == k
    return a, emitted.tolist()


def problem(n, V, dtype, seed, near=0.5):
    g = torch.Generator("cuda").manual_seed(seed)
    T, B = sum(n), len(n)
    logits = 2 * torch.randn(T, V, device="cuda", generator=g)
    p = logits.softmax(-1).to(dtype)
    q = (logits + near * torch.randn(T, V, device="cuda", generator=g)).softmax(-1).to(dtype)
    drafts = torch.multinomial(q.float() + 1e-9, 1, generator=g)[:, 0]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return (cu, drafts.roll(1).tolist(), p, q, torch.rand(T, device="cuda", generator=g), torch.rand(B, device="cuda", generator=g))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,V", [([1], 1), ([1, 2], 2), ([3, 1, 0, 5], 7), ([5] * 6, 1000), ([2, 9, 4], 1031), ([0, 0, 3], 9001), ([4], 33000),
                                 ([3], 20011), ([1] * 70, 64)])
@pytest.mark.parametrize("draft", [True, False])
def test_sampled(n, V, dtype, draft):
    for seed in range(3):
        cu, tokens, p, q, u, pick = problem(n, V, dtype, seed, near=0.2 if seed else 2.0)
        run(cu, tokens, p, q if draft else None, u, pick)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,V", [([1], 1), ([2, 0, 7], 3), ([4, 4, 1], 1029), ([3], 9000), ([13], 50)])
def test_greedy(n, V, dtype):
    for seed in range(3):
        cu, tokens, p, _, _, _ = problem(n, V, dtype, seed)
        best = p.float().argmax(-1).roll(1).tolist()
        tokens = [b if (i + seed) % 4 else t for i, (b, t) in enumerate(zip(best, tokens))]
        run(cu, tokens, p)


def test_greedy_ties_and_odd_values():
    V = 5000
    p = torch.zeros(6, V, device="cuda")
    p[0, 17] = p[0, 4999] = p[0, 18] = 0.25           # the first of equal ones
    p[1] = -math.inf                                  # logits: all the least
    p[2] = math.nan
    p[2, 4000] = -3.0                                 # a number beats NaN
    p[3, :] = -0.0
    p[3, 9] = 0.0                                     # equal to -0
    p[4, 3000] = math.inf
    a, e = run([0, 6], [0, 17, 0, 4000, 0, 3000], p)
    assert a == [5] and e == [17, 0, 4000, 0, 3000, 0]


def test_borders():
    # u q against p where both are equal, next to it, zero and not finite
    V = 8
    tiny = 2.0 ** -24
    rows = [(0.5, 0.25, 0.5), (0.5, 0.25 + 2.0 ** -26, 0.5), (0.5, 0.25 - 2.0 ** -26, 0.5), (0.0, 0.0, 0.0), (0.0, tiny, 0.0), (1.0 - tiny, 1.0, 1.0),
            (0.5, math.nan, 0.5), (0.5, 0.5, math.nan), (0.0, 0.3, 1.0), (0.5, 0.25 + 2.0 ** -25, 0.5)]
    n = len(rows)
    p = torch.full((2 * n, V), 0.1, device="cuda")
    q = torch.full((2 * n, V), 0.1, device="cuda")
    u = torch.zeros(2 * n, device="cuda")
    for i, (x, y, z) in enumerate(rows):
        u[2 * i], p[2 * i, 3], q[2 * i, 3] = x, y, z
    a, _ = run([2 * i for i in range(n + 1)], [3] * (2 * n), p, q, u, torch.rand(n, device="cuda"))
    # fp32 holds 0.25 + 2^-26 as 0.25 (its step there is 2^-25, and a half goes to the even one): 0.25 < 0.25 is not so;
    # (1 - 2^-24) 1 < 1 is
    assert a == [0, 0, 0, 0, 1, 1, 0, 0, 1, 1]


def test_what_is_left():
    # all mass gone: p itself; no mass at all: -1; drafts outside the vocabulary; the last row's draft is not read
    V = 3000
    p, q = torch.zeros(10, V, device="cuda"), torch.full((10, V), 1.0, device="cuda")
    p[0, 5] = p[2, 2999] = 0.5
    p[3, :] = math.nan
    p[6, 7] = 0.25
    p[8] = -1.0
    q[1::2] = math.nan
    tokens = [0, 5, 0, -1, 0, 7, 0, V, 0, 1 << 30]
    u = torch.full((10,), 0.9, device="cuda")
    a, e = run([0, 2, 4, 6, 8, 10], tokens, p, q, u, torch.tensor([0.3, 0.999, 0.5, 0.5, 0.0], device="cuda"))
    assert a == [0] * 5 and e == [5, -1, 2999, -1, -1, -1, 7, -1, -1, -1]
    p[9], u[8] = 0, 0.0
    p[9, 11], tokens[9], p[8, 4] = 2.0, 4, 0.1
    a, e = run([8, 10], tokens, p, q, u, torch.tensor([0.5], device="cuda"))
    assert a == [1] and e[8:] == [4, 11]


@pytest.mark.parametrize("pick", [0.0, 1.0 - 2.0 ** -24, 1.0, -1.0, math.nan, 2.0 ** -32, math.inf])
def test_the_point_at_its_ends(pick):
    V = 4097
    p = torch.zeros(1, V, device="cuda")
    p[0, 1], p[0, 2000], p[0, V - 1] = 0.25, 2.0 ** -42, 0.5
    p[0, 9] = 2.0 ** -43                              # counts as nothing
    _, e = run([0, 1], [0], p, None, torch.zeros(1, device="cuda"), torch.tensor([pick], device="cuda"))
    assert e[0] == (V - 1 if pick > 0.5 else 1)


def test_rows_as_they_lie():
    # row strides, rows that start anywhere, one distribution for all rows, requests out of the front of the buffers
    V = 777
    cu, tokens, p, q, u, pick = problem([3, 4], V, torch.bfloat16, 5)
    wide = torch.full((7, V + 6), 9.0, device="cuda").bfloat16()
    wide[:, 3:3 + V] = p
    run(cu, tokens, wide[:, 3:3 + V], q, u, pick)
    run(cu, tokens, p, q[:1].expand(7, V), u, pick)
    run([2, 2, 6], tokens, p, q, u, pick)


def test_distribution():
    # the tokens emitted are distributed as the target says, whatever drafted them
    V, B = 6, 20000
    g = torch.Generator("cuda").manual_seed(0)
    p = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1], device="cuda").expand(2 * B, V)
    q = torch.tensor([0.3, 0.1, 0.3, 0.1, 0.1, 0.1], device="cuda").expand(2 * B, V)
    d = torch.multinomial(q[0], 2 * B, True, generator=g).int()
    cu = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda")
    accepted, emitted = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(2 * B, dtype=torch.int32, device="cuda")
    fk.fk_verify(cu, d, p, accepted, emitted, draft=q, accept=torch.rand(2 * B, device="cuda", generator=g),
                 pick=torch.rand(B, device="cuda", generator=g))
    got = torch.bincount(emitted[::2].long(), minlength=V).double() / B
    # five standard deviations of a share: 5 sqrt(0.25 / B)
    assert float((got - p[0].double()).abs().max()) < 5 * math.sqrt(0.25 / B)


def test_many_requests():
    # more requests than one dimension of a grid holds
    B, V = 40000, 40
    g = torch.Generator("cuda").manual_seed(1)
    p = torch.rand(B, V, device="cuda", generator=g)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(B, dtype=torch.int32, device="cuda")
    accepted, emitted = torch.empty_like(tokens), torch.empty_like(tokens)
    fk.fk_verify(cu, tokens, p, accepted, emitted)
    assert torch.equal(emitted.long(), p.argmax(-1)) and not bool(accepted.any())
    fk.fk_verify(cu, tokens, p, accepted, emitted, accept=torch.zeros(B, device="cuda"), pick=torch.zeros(B, device="cuda"))
    assert not bool(emitted.any())


def test_on_another_stream():
    cu, tokens, p, q, u, pick = problem([3, 4, 1], 30000, torch.float32, 8)
    side = torch.cuda.Stream()
    size = fk.verify_workspace(i32(cu), p).numel()
    accepted, emitted = i32([-9] * 3), i32([-9] * 8)
    args = (i32(cu), i32(tokens), p, accepted, emitted)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stall(side)
    fk.fk_verify(*args, draft=q, accept=u, pick=pick, stream=side)
    assert Bystanders([size]).untouched()
    a, e, _ = ref.verify(cu, tokens, p, q, u.tolist(), pick.tolist(), [0] * 3)
    assert accepted.tolist() == a and emitted.tolist() == [e[r] for r in range(8)]


def test_captured():
    cu, tokens, p, q, u, pick = problem([3, 4, 1], 5000, torch.float32, 9)
    c, t = i32(cu), i32(tokens)
    out = [i32([0] * 3), i32([0] * 8)]
    ws = fk.verify_workspace(c, p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fk.fk_verify(c, t, p, *out, draft=q, accept=u, pick=pick, ws=ws)
    for seed in range(3):
        g = torch.Generator("cuda").manual_seed(seed)
        u.copy_(torch.rand(8, device="cuda", generator=g))
        pick.copy_(torch.rand(3, device="cuda", generator=g))
        ws.fill_(255)
        graph.replay()
        a, e, _ = ref.verify(cu, tokens, p, q, u.tolist(), pick.tolist(), [0] * 3)
        assert out[0].tolist() == a and out[1].tolist() == [e[r] for r in range(8)]
