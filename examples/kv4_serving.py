"""A small serving loop on the 4-bit cache: codebooks learned by k-means from a
sample, ragged prompts, then single tokens, with the attention's error against
the unquantised rows.

    python examples/kv4_serving.py [--steps 8]

Then one prompt is continued in four ways: its pages are shared and read once
for all, each step brings drafts, and those that the target refuses are taken
back.

There is no model here: queries, keys and values are drawn at random, keys
with channels that stand out as they do after rotary embeddings.  The error
is that of 4 bits, shown for the learned codebooks and for 16 equal steps.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import exact_lloyd_means_amd as fk  # noqa: E402

B, Hq, H, D, P = 6, 32, 8, 128, 64


class Source:
    """Seeded rows of the shapes that a layer's projections give."""

    def __init__(self, seed=0):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.channels = torch.exp(0.5 * torch.randn(H, D, device="cuda", generator=self.g))

    def __call__(self, n):
        q, k, v = (torch.randn(n, h, D, device="cuda", generator=self.g) for h in (Hq, H, H))
        # independent values, as in most heads: keys keep their channels' magnitudes
        return q.bfloat16(), (k * self.channels).bfloat16(), v.bfloat16()


def reference(q, rows, cu, lens):
    """Attention over the unquantised rows of each request, in fp32."""
    out = torch.empty(q.shape, device="cuda")
    for b in range(B):
        k, v = (torch.cat(r).float().repeat_interleave(Hq // H, 1) for r in rows[b])
        x = q[cu[b]:cu[b + 1]].float()
        s = torch.einsum("qhd,khd->hqk", x, k) / math.sqrt(D)
        pos = torch.arange(lens[b] - len(x), lens[b], device="cuda")
        s.masked_fill_(torch.arange(lens[b], device="cuda") > pos[:, None], -math.inf)
        out[cu[b]:cu[b + 1]] = torch.einsum("hqk,khd->qhd", s.softmax(-1), v)
    return out


def serve(codebook, steps, seed=1):
    """Prompts and `steps` single tokens; the relative error of every step."""
    source, errors = Source(seed), []
    cache = fk.KV4Cache(200, P, H, D, codebook, max_requests=B, max_len=2048)
    rows, lens = [([], []) for _ in range(B)], [0] * B
    for step in range(1 + steps):
        new = [37, 800, 1, 256, 511, 64] if step == 0 else [1] * B
        total = sum(new)
        cache.plan(torch.tensor(new, dtype=torch.int32, device="cuda"), total)
        q, k, v = source(total)
        cache.append(k, v)
        out = cache.attend(q, max(new))
        cu = [sum(new[:b]) for b in range(B + 1)]
        for b in range(B):
            rows[b][0].append(k[cu[b]:cu[b + 1]])
            rows[b][1].append(v[cu[b]:cu[b + 1]])
            lens[b] += new[b]
        want = reference(q, rows, cu, lens)
        errors.append(float((out.float() - want).norm() / want.norm()))
    assert cache.lens.tolist() == lens and cache.status.tolist()[2:] == [0, 0]
    free = int(cache.free_count)
    cache.release(torch.tensor([1, 4], device="cuda"))
    assert int(cache.free_count) - free == sum(-(-lens[b] // P) for b in (1, 4))
    return errors


def continued(codebook, steps, samples=4, drafts=3, vocabulary=5000, seed=2):
    """A prompt continued in `samples` ways by `steps` steps of drafts; pages in
    use, pages that rows of their own would take, tokens a step and sample."""
    source, turns = Source(seed), fk.rope_turns(D)
    cache = fk.KV4Cache(200, P, H, D, codebook, max_requests=samples, max_len=2048)
    i32 = dict(dtype=torch.int32, device="cuda")
    prompt, kept = 900, 0

    def step(new, total, max_q, shared=None):
        cache.plan(new, total)
        q, k, v = source(total)
        cache.rotate(q, k, turns)
        cache.append(k, v)
        return cache.attend(q, max_q, shared=shared)
    step(torch.tensor([prompt] + [0] * (samples - 1), **i32), prompt, prompt)
    cache.fork(torch.arange(1, samples, **i32), torch.zeros(samples - 1, **i32))
    shared = torch.tensor([0, samples], **i32), torch.tensor([prompt // P * P], **i32)
    new, total = torch.full((samples,), 1 + drafts, **i32), samples * (1 + drafts)
    for _ in range(steps):
        step(new, total, 1 + drafts, shared)
        # distributions such as a model and a small model that drafts for it give
        logits = torch.randn(total, vocabulary, device="cuda", generator=source.g)
        near = logits + 0.5 * torch.randn(total, vocabulary, device="cuda", generator=source.g)
        target, draft = logits.softmax(-1), near.softmax(-1)
        tokens = torch.multinomial(draft, 1, generator=source.g)[:, 0].int().roll(1)
        accepted, _ = cache.verify(tokens, target, draft, torch.rand(total, device="cuda", generator=source.g),
                                   torch.rand(samples, device="cuda", generator=source.g))
        kept += int(accepted.sum()) + samples
    lens = cache.lens.tolist()
    assert sum(lens) == samples * prompt + kept and cache.status.tolist()[2:] == [0, 0]
    alone = sum(-(-n // P) for n in lens)
    return 200 - int(cache.free_count), alone, kept / (steps * samples)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    steps = ap.parse_args().steps
    _, k, v = Source(1)(4096)
    learned = fk.learn_codebook(k, v)
    even = torch.linspace(-1, 1, 16, device="cuda").half().expand(2, H, 16).contiguous()
    for name, codebook in (("16 equal steps", even), ("k-means", learned)):
        e = serve(codebook, steps)
        print(f"{name:15s} error of the prompts {e[0]:.4f}, of single tokens "
              f"{sum(e[1:]) / max(1, len(e) - 1):.4f}")
    used, alone, tokens = continued(learned, max(1, steps))
    print(f"one prompt in four ways: {used} pages instead of {alone}, {tokens:.2f} tokens a step")


if __name__ == "__main__":
    main()
