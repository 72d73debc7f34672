"""The 4-bit cache on another stream than the current one: workspaces, slots
and results belong to the stream that uses them."""
import torch
import pytest

import exact_lloyd_means_amd as fk
import kv4_ref as ref
from test_gpu_streams import Bystanders, stall

pytestmark = pytest.mark.gpu
H, D, P, B = 2, 128, 64, 3


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def test_workspace_of_the_plan():
    # two launches: the second reads what the first left in the workspace
    side = torch.cuda.Stream()
    i32 = dict(dtype=torch.int32, device="cuda")
    n, cap = 6000, 20000

    def outputs():
        return [torch.full((n, 4), -1, **i32), torch.empty(n, **i32), torch.empty(n + 1, **i32), torch.empty(cap, **i32),
                torch.empty(cap, **i32), torch.empty(1, **i32), torch.empty(4, **i32)]
    ctx, new = torch.zeros(n, **i32), torch.full((n,), 3, **i32)
    free, count = torch.arange(n, **i32), torch.tensor([n], **i32)
    want, got = outputs(), outputs()
    fk.fk_kv_plan(ctx, new, P, free, count, *want)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stall(side)
    fk.fk_kv_plan(ctx, new, P, free, count, *got, stream=side)
    assert Bystanders([4 * (n + 1)]).untouched()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("handle", [False, True])
def test_workspace_of_the_attention(handle):
    # shares with a join: the sums lie in the workspace between two launches
    side = torch.cuda.Stream()
    g = torch.Generator("cuda").manual_seed(1)
    pages = 40
    codes = torch.randint(0, 256, (pages, H, 2, P // 32, 16 * D), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.rand(pages, H, 2, P, device="cuda", generator=g).bfloat16()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1).repeat(1, 10)
    q = torch.randn(3, 8, D, device="cuda", generator=g).bfloat16()
    cu, seq = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [pages * P]))
    out = [torch.zeros_like(q) for _ in range(2)]
    args = (q, cu, seq, table, ref.codebook(H).cuda(), codes, scales)
    fk.fk_kv4_attention(*args, out[0], 3)
    size = fk.kv4_attention_workspace(q, seq, codes, 3).numel()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stall(side)
    fk.fk_kv4_attention(*args, out[1], 3, stream=side.cuda_stream if handle else side)
    assert Bystanders([size]).untouched()
    assert torch.equal(out[0], out[1])


def test_a_serving_loop_on_a_side_stream():
    # what a step made is dropped while the side stream is still busy
    side = torch.cuda.Stream()
    g = torch.Generator().manual_seed(2)
    cb = ref.codebook(H, 1).cuda()
    steps = []
    for new in ([300, 5, 70], [1, 1, 1], [1, 1, 1]):
        T = sum(new)
        steps.append([torch.tensor(new, dtype=torch.int32, device="cuda")] +
                     [torch.randn(T, h, D, generator=g).bfloat16().cuda() for h in (8, H, H)])

    def loop(stream, before=lambda: None, after=lambda n: None):
        cache = fk.KV4Cache(60, P, H, D, cb, B, 2048)
        row = torch.tensor([1], device="cuda")
        torch.cuda.synchronize()
        outs = []
        for i, (new, q, k, v) in enumerate(steps):
            before()
            cache.plan(new, len(q), stream=stream)
            cache.append(k, v, stream=stream)
            out = cache.attend(q, int(max(300 if i == 0 else 1, 1)), stream=stream)
            outs.append(out.clone() if stream is None else None)
            if stream is not None:
                with torch.cuda.stream(stream):
                    outs[-1] = out.clone()
            del out
            after(len(q))
        cache.release(row, stream=stream)
        torch.cuda.synchronize()
        return outs, cache
    want, plain = loop(None)
    torch.cuda.empty_cache()
    by = []
    got, cache = loop(side, lambda: stall(side), lambda n: by.append(Bystanders([4 * n, n * 8 * D * 2])))
    assert all(b.untouched() for b in by)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for name in ("block_table", "free_count", "lens", "codes", "scales"):
        assert torch.equal(getattr(cache, name), getattr(plain, name)), name


@pytest.mark.parametrize("busy", ["current", "side"])
@pytest.mark.parametrize("handle", [False, True])
def test_codebook_learned_on_a_side_stream(handle, busy):
    # samples still being made by the current stream, or the side stream behind
    # with other work: the result is the same, and ready for the current stream
    side = torch.cuda.Stream()
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn(500, H, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    want = fk.learn_codebook(k, v, iters=5)
    torch.cuda.synchronize()
    stall(side if busy == "side" else torch.cuda.current_stream())
    k2, v2 = k * 2, v * 2                            # the same over each row's largest
    got = fk.learn_codebook(k2, v2, iters=5, stream=side.cuda_stream if handle else side)
    del k2, v2
    Bystanders([500 * H * D * 2])
    assert torch.equal(got, want)
