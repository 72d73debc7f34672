"""KV4Cache and learn_codebook: a serving loop against the functions' own
reference, pages returned and taken again, the example."""
import math
import os
import subprocess
import sys

import pytest
import torch

import exact_lloyd_means_amd as fk
import kv4_ref as ref
import oracle

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def test_codebook_is_that_of_k_means():
    g = torch.Generator().manual_seed(0)
    T, H, D = 300, 3, 64
    k, v = (torch.randn(T, H, D, generator=g).bfloat16().cuda() for _ in range(2))
    k[5] = 0                                        # a row of zeros
    cb = fk.learn_codebook(k, v, iters=12)
    assert cb.shape == (2, H, 16) and cb.dtype == torch.float16
    assert bool((cb.diff(dim=-1) >= 0).all()) and bool((cb.abs() <= 1).all())
    # lock-step Lloyd in fp64 from the same levels
    x = torch.stack((k, v)).float()
    x = (x / x.abs().amax(-1, keepdim=True).clamp(min=1e-38)).permute(0, 2, 1, 3).reshape(2 * H, T * D, 1)
    C = torch.linspace(-1, 1, 16).view(1, 16, 1).repeat(2 * H, 1, 1)
    xs = x.cpu().contiguous().numpy()
    for _ in range(12):
        lab, _, _ = oracle.assign(xs, C.numpy(), fmt_x="f32", fmt_c="f32")
        _, c, _ = oracle.update(xs, lab.reshape(2 * H, -1), C.numpy(), fmt_x="f32", fmt_c="f32")
        C = torch.from_numpy(c).float()
    # points at the middle of two levels may fall to either side in fp32: a
    # centroid of T D / 16 = 1200 points moves by far less than this
    assert float((cb.cpu().float().view(2 * H, 16) - C.view(2 * H, 16).sort(-1).values).abs().max()) < 2e-3


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_serving_loop(dtype):
    B, Hq, H, D, P, pages = 5, 8, 2, 64, 32, 40
    g = torch.Generator().manual_seed(3)
    cb = ref.codebook(H, 2)
    cache = fk.KV4Cache(pages, P, H, D, cb.cuda(), B, 300, dtype=dtype)
    lens = [0] * B
    for step, new in enumerate(([40, 0, 33, 100, 1], [1] * 5, [1, 20, 1, 0, 1], [3, 3, 3, 3, 3])):
        T = sum(new) + 2                             # two tokens of padding
        q = torch.randn(T, Hq, D, generator=g).to(dtype)
        k, v = (torch.randn(T, H, D, generator=g).to(dtype) for _ in range(2))
        slots, positions, cu = cache.plan(torch.tensor(new, dtype=torch.int32, device="cuda"), T)
        cache.append(k.cuda(), v.cuda())
        lse = torch.empty(T, Hq, device="cuda")
        out = cache.attend(q.cuda(), max(new), lse=lse)
        torch.cuda.synchronize()
        lens = [a + b for a, b in zip(lens, new)]
        assert cache.lens.tolist() == lens
        pos = [i for a, n in zip(lens, new) for i in range(a - n, a)] + [-1, -1]
        assert positions.tolist() == pos and slots.tolist()[-2:] == [-1, -1]
        n = sum(new)
        want = ref.attention(q[:n], cu.cpu(), lens, cache.block_table.cpu(), cb, cache.codes.cpu(),
                             cache.scales.cpu(), 1 / math.sqrt(D), True, 0)
        tol, tol_lse = ref.attention_tolerance(*want, D, dtype)
        assert bool(((out[:n].cpu().double() - want[0]).abs() <= tol).all())
        assert bool(((lse[:n].cpu().double() - want[1]).abs() <= tol_lse).all())
    # the cache holds what was appended: every page is named once
    used = cache.block_table[cache.block_table >= 0].tolist()
    assert len(set(used)) == len(used) == pages - int(cache.free_count)
    cache.release(torch.tensor([3, 0], device="cuda"))
    left = cache.free_pages[:int(cache.free_count)].tolist()
    held = cache.block_table[cache.block_table >= 0].tolist()
    assert sorted(left + held) == list(range(pages))
    assert cache.lens.tolist() == [0, lens[1], lens[2], 0, lens[4]]
    # a request larger than what is left
    cache.plan(torch.tensor([299, 270, 270, 299, 270], dtype=torch.int32, device="cuda"), 1408)
    assert int(cache.free_count) == 0 and cache.status.tolist()[2] > 0


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "kv4_serving.py"), "--steps", "2"],
                       capture_output=True, text=True, timeout=110, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [l for l in r.stdout.splitlines() if "error of the prompts" in l]
    errors = [float(l.split("prompts ")[1].split(",")[0]) for l in lines]
    assert len(errors) == 2 and errors[1] < errors[0]    # learned levels beat equal ones
