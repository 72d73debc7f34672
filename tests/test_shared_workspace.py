"""Workspaces of fk_kv4_attention_shared, on the CPU: one for the largest step does
for all smaller ones.  What a call takes is what it asks for when it gets less."""
import random
import re
import struct

import pytest

import exact_lloyd_means_amd as fk

CACHE, ATTN, FAKE = struct.Struct("@PPPqiiii"), struct.Struct("@qqiiqqqPPPPfiiPP"), 0x10000


def cache(H, D):
    return CACHE.pack(FAKE, FAKE, FAKE, 1000, 64, H, D, fk.FK_BF16)


def size(B, T, Hq, H, D, max_q, groups):
    return fk.lib.fk_kv4_attn_shared_workspace_bytes(cache(H, D), B, T, Hq, max_q, groups)


def takes(B, T, Hq, H, D, max_q, groups, pages, window=0):
    """Bytes without which the call is refused; it is never launched."""
    a = ATTN.pack(B, T, Hq, max_q, pages, Hq * D, D, FAKE, FAKE, FAKE, FAKE, 0.1, 1, window, FAKE, 0)
    assert fk.lib.fk_kv4_attention_shared(cache(H, D), a, groups, FAKE, FAKE, FAKE, 1, None) == fk.FK_EWORKSPACE
    return int(re.search(r"needs (\d+)", fk.lib.fk_last_error().decode())[1])


HEADS = [(8, 8, 64), (32, 8, 128), (64, 8, 128), (32, 1, 128), (20, 1, 64), (48, 1, 128), (16, 16, 128), (96, 4, 64), (16, 1, 256), (8, 2, 256),
         (32, 16, 256), (9, 3, 128), (40, 2, 64)]


@pytest.mark.parametrize("Hq,H,D", HEADS)
def test_more_groups_need_no_less(Hq, H, D):
    for B, T, q in ((64, 64, 1), (600, 600, 1), (64, 192, 3), (300, 900, 3), (16, 800, 50), (40, 4000, 100), (9000, 9000, 1)):
        last = 0
        for groups in range(1, min(B, 700) + 1):
            n = size(B, T, Hq, H, D, q, groups)
            assert n >= last, (B, T, q, groups)
            last = n


@pytest.mark.parametrize("Hq,H,D", HEADS)
def test_more_requests_and_tokens_need_no_less(Hq, H, D):
    most = 48 if D < 256 else 16
    for q in (1, 2, 3, 5, 8, 16):
        if q * (Hq // H) > most:
            continue
        for groups in (1, 3, 30):
            by_requests = [size(B, 5000, Hq, H, D, q, groups) for B in range(groups, 900, 7)]
            assert by_requests == sorted(by_requests)
            by_tokens = [size(200, T, Hq, H, D, q, groups) for T in [*range(1, 100), *range(100, 9000, 61)]]
            assert by_tokens == sorted(by_tokens)
            by_q = [size(200, 300, Hq, H, D, x, groups) for x in range(1, most // (Hq // H) + 1)]
            assert by_q == sorted(by_q)


@pytest.mark.parametrize("Hq,H,D", HEADS)
def test_it_does_for_smaller_calls(Hq, H, D):
    r = random.Random(Hq * D + H)
    G, most, shared = Hq // H, 48 if D < 256 else 16, 0
    for _ in range(1500):
        q = r.choice([1, 1, 2, 3, 4, 6, 9, 16, 40, 100])
        B = int(2 ** r.uniform(0, 10))
        groups = r.randrange(1, B + 1) if r.random() < 0.3 else r.randrange(1, min(B, 20) + 1)
        T = r.randrange(1, B * q + 1)
        have = size(B, T, Hq, H, D, q, groups)
        for _ in range(3):
            b = r.randrange(1, B + 1)
            g = r.randrange(1, min(b, groups) + 1)
            t, max_q = (r.randrange(1, T + 1), r.randrange(1, q + 1)) if G * min(q, T) <= most else (T, q)
            pages = r.choice([1, 8, 40, 300, 2000, 20000])
            if b * pages * 2 > 2 ** 31 - 1:
                continue
            need = takes(b, t, Hq, H, D, max_q, g, pages, r.choice([0, 0, 100, 5000]))
            shared += need > 256
            assert need <= have, (B, T, q, groups, b, t, max_q, g, pages)
    assert shared > 500
