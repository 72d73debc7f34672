"""fk_kv_plan with far more new tokens than slots: tables are filled page by
page, in a time that does not follow the tokens."""
import random

import pytest
import torch

import exact_lloyd_means_amd as fk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def definition(ctx, new, P, M, free, cap):
    """Table entries, slots and positions from the definition, page by page."""
    top, left, table, slots, pos = 2 ** 31 - 1, len(free), {}, [], []
    wanted = lost = 0
    for b, (c, f) in enumerate(zip(ctx, new)):
        held, got = -(-c // P), 0
        for p in range(held, min(-(-min(c + f, top) // P), M)):
            wanted += 1
            table[b, p] = free[left - 1] if left > 0 else -1
            got += left > 0
            left -= left > 0
        lost += max(0, c + f - max(c, (min(held, M) + got) * P))
        for i in range(c, c + min(f, max(0, cap - len(slots)))):
            page = table.get((b, i // P), -1) if i // P >= held else 1000 + i // P if i // P < M else -1
            slots.append(page * P + i % P if page >= 0 else -1)
            pos.append(i)
    taken = len(free) - left
    return table, slots, pos, [min(sum(new), top), taken, wanted - taken, min(lost, top)]


def plan(ctx, new, P, M, nfree, cap):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    B, free = len(ctx), list(range(5, 5 + nfree))
    before = torch.full((B, M), -7, dtype=torch.int32)
    for b, c in enumerate(ctx):
        held = min(-(-c // P), M)
        before[b, :held] = 1000 + torch.arange(held)
    out = [before.cuda(), i32([0] * B), i32([0] * (B + 1)), i32([-5] * cap), i32([-5] * cap), i32([0]), i32([0] * 4)]
    args = [i32(ctx), i32(new), P, i32(free), i32([nfree])]
    fk.fk_kv_plan(*args, *out)
    torch.cuda.synchronize()
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    fk.fk_kv_plan(*args, *out)
    t[1].record()
    torch.cuda.synchronize()
    table, slots, pos, status = definition(ctx, new, P, M, free, cap)
    for (b, p), page in table.items():
        before[b, p] = page
    assert torch.equal(out[0].cpu(), before)
    assert out[3].tolist() == slots + [-1] * (cap - len(slots)) and out[4].tolist() == pos + [-1] * (cap - len(pos))
    assert out[6].tolist() == status
    return t[0].elapsed_time(t[1])


@pytest.mark.parametrize("B,cap", [(16, 8), (16, 0), (1000, 5000), (5000, 100)])   # one launch, and two
def test_time_follows_slots_and_pages(B, cap):
    r = random.Random(B)
    ctx, M = [r.choice([0, 1, 1024, 5000]) for _ in range(B)], 262144 // B + 8
    new = [r.choice([0, (M - 8) * 1024]) for _ in range(B)]        # 2^27 tokens, 2^17 pages
    # a workgroup that walked the tokens would take most of a second
    assert plan(ctx, new, 1024, M, 131072 - 77, cap) < 50


@pytest.mark.parametrize("B", [3, 4500])
def test_sums_that_saturate(B):
    # the table ends long before the tokens do
    ctx, new = [0, 64, 7] * (B // 3), [2 ** 31 - 1, 2 ** 31 - 65, 5] * (B // 3)
    assert plan(ctx, new, 32, 40, 9, 100) < 50
