"""KV4Cache after a step that found no page for some of its tokens."""
import math

import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref

pytestmark = pytest.mark.gpu
H, Hq, D, P = 1, 2, 64, 32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


class Loop:
    """A cache beside the rows it should hold; new tokens are drawn at random."""

    def __init__(self, pages, B, max_len):
        self.cb = ref.codebook(H, 0)
        self.cache = fk.KV4Cache(pages, P, H, D, self.cb.cuda(), B, max_len)
        self.held = [0] * B
        self.g = torch.Generator().manual_seed(0)

    def step(self, new):
        """Plans, appends and attends; the number of tokens kept of each request."""
        T, c = sum(new), self.cache
        slots, positions, cu = c.plan(torch.tensor(new, dtype=torch.int32, device="cuda"), T)
        assert positions.tolist() == [h + i for h, n in zip(self.held, new) for i in range(n)]
        q, k, v = (torch.randn(T, h, D, generator=self.g).bfloat16() for h in (Hq, H, H))
        c.append(k.cuda(), v.cuda())
        seq = [h + n for h, n in zip(self.held, new)]
        out = c.attend(q.cuda(), max(new))
        want = ref.attention(q, cu.cpu(), seq, c.block_table.cpu(), self.cb, c.codes.cpu(), c.scales.cpu(),
                             1 / math.sqrt(D), True, 0)
        tol, _ = ref.attention_tolerance(*want, D, torch.bfloat16)
        assert bool(((out.cpu().double() - want[0]).abs() <= tol).all())
        got, at, slots = [], 0, slots.tolist()
        for n in new:
            mine = slots[at:at + n]
            at += n
            kept = sum(s >= 0 for s in mine)
            assert all(s >= 0 for s in mine[:kept])              # a prefix
            got.append(kept)
        assert c.status.tolist()[3] == T - sum(got)              # every token without a slot is told
        self.held = [h + n for h, n in zip(self.held, got)]
        assert c.lens.tolist() == self.held
        return got

    def release(self, b):
        self.cache.release(torch.tensor([b], device="cuda"))
        self.held[b] = 0


def test_a_page_is_given_once_there_is_one():
    s = Loop(pages=3, B=2, max_len=320)
    assert s.step([64, 32]) == [64, 32]
    assert s.step([1, 0]) == [0, 0]                              # the list is spent
    assert s.step([1, 1]) == [0, 0]
    s.release(1)
    assert s.step([1, 0]) == [1, 0]
    assert s.step([31, 0]) == [31, 0]
    assert s.step([1, 0]) == [0, 0]
    assert s.step([0, 5]) == [0, 0]


def test_part_of_a_prompt():
    s = Loop(pages=5, B=3, max_len=320)
    assert s.step([40, 200, 7]) == [40, 96, 0]
    s.release(0)
    assert s.step([0, 40, 7]) == [0, 40, 0]                      # the two pages go to request 1
    s.release(1)
    assert s.step([33, 0, 70]) == [33, 0, 70]


def test_the_end_of_the_table():
    s = Loop(pages=20, B=2, max_len=64)
    assert s.step([60, 3]) == [60, 3]
    assert s.step([9, 1]) == [4, 1]
    assert s.step([1, 1]) == [0, 1]
    s.release(0)
    assert s.step([64, 0]) == [64, 0]
    assert int(s.cache.free_count) == 17


@pytest.mark.parametrize("B", [40, 5000])      # one and two launches
@pytest.mark.parametrize("count", [0, 30, 100000])
def test_kept_lengths_are_those_with_a_page(B, count):
    import random
    r = random.Random(B + count)
    page, M = 32, 4
    ctx = [r.choice([0, 5, 32, 100, 128]) for _ in range(B)]
    new = [r.choice([0, 1, 40, 90]) for _ in range(B)]
    held = [-(-c // page) for c in ctx]
    table = [[1000 + p if p < h else -1 for p in range(M)] for h in held]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = [i32(table), i32([0] * B), i32([0] * (B + 1)), i32([0] * (sum(new) + 1)), None, i32([0]), i32([0] * 4)]
    kept, free = i32([-5] * B), list(range(2000, 2000 + count))
    fk.fk_kv_plan(i32(ctx), i32(new), page, i32(free), i32([count]), *out, kept_lens=kept)
    want = ref.plan(ctx, new, page, table, free, count, sum(new) + 1)
    assert out[0].tolist() == table and out[1].tolist() == want["seq"]
    slots, cu = want["slots"], want["cu"]
    assert kept.tolist() == [c + sum(s >= 0 for s in slots[a:b]) for c, a, b in zip(ctx, cu, cu[1:])]
